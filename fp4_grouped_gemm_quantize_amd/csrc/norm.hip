// norm.hip -- root-mean-square norm of a residual stream with the residual's
// addition and an 8-bit output, and its gradient, for gfx950.
//
//   h = x + res,  r = 1 / sqrt(sum h^2 / H + eps),  y = h (w + o) r
//   g = dy (w + o),  dx = dh + r g - h r^3 (sum g h) / H,  dw = sum over rows of dy h r
//
// Both are HBM-bound streams: a row is read once, held in registers between its sums
// and its outputs, and written once.  Forward a workgroup per row (64, 256 or 1024 threads by the row's
// length, up to four vectors of 8 elements a thread), or per several rows where there are more than
// 2^28 threads' worth; backward up to 512 workgroups (64 to 1024 threads, up to two vectors each) that walk the rows with
// the weight and its gradient's sums in registers.
// 8192 x 4096 bf16 with residual and block-128 codes 58 us (302 MB, 5.2 TB/s; the three passes of
// separate kernels move 1.4 times as much); the gradient of 8192 x 7168 99 us (470 MB, 4.8 TB/s); 64 x
// 7168 8.5 us, of which 5.8 on the device: the launch, one trip to memory, one barrier.
#include "fp8_encode.h"
#include "mxg_device.h"
#include "mxg_internal.h"

#include <type_traits>

namespace mxg {

namespace {

constexpr int kPlain = 0, kRowwise = 1, kMX = 2, kBlock = 3;  // mxg_norm_format

struct NormArgs {
    const void* x;
    const void* res;
    const void* w;
    float w_add, eps;
    int64_t T, H;
    void* h;
    uint16_t* y;
    uint8_t* q;
    void* scales;
    bool w32;
};

// Elements 8 v .. 8 v + 7 of a row of fp32 or bf16.
template <bool F32>
__device__ __forceinline__ void load8(const void* row, int64_t v, float* f) {
    if constexpr (F32) {
        const float4 a = reinterpret_cast<const float4*>(row)[2 * v], b = reinterpret_cast<const float4*>(row)[2 * v + 1];
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
        unpack8(reinterpret_cast<const uint4*>(row)[v], f);
    }
}
__device__ __forceinline__ uint4 pack8_bf16(const float* f) {
    return make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]), f32x2_to_bf16x2(f[4], f[5]),
                      f32x2_to_bf16x2(f[6], f[7]));
}
template <bool F32>
__device__ __forceinline__ void store8(void* row, int64_t v, const float* f) {
    if constexpr (F32) {
        reinterpret_cast<float4*>(row)[2 * v] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(row)[2 * v + 1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        reinterpret_cast<uint4*>(row)[v] = pack8_bf16(f);
    }
}
// The same of the gradient's workspace, which lies on 4 bytes (a 16-byte access needs no more of the memory path).
typedef float f4_on4 __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ void load8_ws(const float* row, int64_t v, float* f) {
    const f4_on4 a = reinterpret_cast<const f4_on4*>(row)[2 * v], b = reinterpret_cast<const f4_on4*>(row)[2 * v + 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
}
__device__ __forceinline__ void store8_ws(float* row, int64_t v, const float* f) {
    reinterpret_cast<f4_on4*>(row)[2 * v] = f4_on4{f[0], f[1], f[2], f[3]};
    reinterpret_cast<f4_on4*>(row)[2 * v + 1] = f4_on4{f[4], f[5], f[6], f[7]};
}
template <bool F32>
__device__ __forceinline__ void* row_at(void* p, int64_t e) {
    return static_cast<uint8_t*>(p) + e * (F32 ? 4 : 2);
}
template <bool F32>
__device__ __forceinline__ const void* row_at(const void* p, int64_t e) {
    return static_cast<const uint8_t*>(p) + e * (F32 ? 4 : 2);
}

__device__ __forceinline__ void load_weight8(const NormArgs& a, int64_t v, float* f) {
    if (a.w32) load8<true>(a.w, v, f);
    else load8<false>(a.w, v, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += a.w_add;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
    return v;
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, kWave));
    return v;
}

// Sum over the workgroup, in a fixed order; s holds a word per wave and is used again only
// after another barrier.
template <int NT>
__device__ __forceinline__ float block_sum(float v, float* s) {
    v = wave_sum(v);
    if constexpr (NT > kWave) {
        if ((threadIdx.x & (kWave - 1)) == 0) s[threadIdx.x / kWave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < NT / kWave; ++i) v += s[i];
    }
    return v;
}
__device__ __forceinline__ float inverse_rms(float sum, int64_t H, float eps) {
    return 1.0f / sqrtf(sum / (float)H + eps);
}

// The fp32-scaled formats encode u = h (weight + offset) under amax |u| / 448 and store that
// times r as the scale: r is common to a row, so the codes are those of y under its own
// scale with two roundings fewer (of y and of its maximum), and a row's largest |u| is found
// beside its sum of squares.  Where the scale itself is 0 (r or all of u) or r is NaN, so is
// what the codes are taken under.
struct Scale {
    float of_y, of_u;
};
__device__ __forceinline__ Scale scale_of(float top, float r) {
    const float s = top / 448.0f, of_y = s * r;  // IEEE binary32 division
    return {of_y, of_y == 0.0f || r != r ? of_y : s};
}

// 8 values u = h (weight + offset) (vector v of row t) out, as y = u r: bf16 and codes.  Every lane of
// the wave calls it, with `in` false (and u 0) past the row's end; row: the rowwise format's scale.
template <int FMT>
__device__ __forceinline__ void put8(const NormArgs& a, int64_t t, int64_t v, bool in, const float* u, float r,
                                     const Scale& row) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = u[i] * r;
    if (in && a.y) reinterpret_cast<uint4*>(a.y + t * a.H)[v] = pack8_bf16(y);
    if constexpr (FMT == kRowwise) {
        if (in) *reinterpret_cast<uint2*>(a.q + t * a.H + v * 8) = encode8(u, row.of_u);
    } else if constexpr (FMT == kBlock) {
        const Scale s = scale_of(amax_of16(amax8(u)), r);
        if (in) {
            *reinterpret_cast<uint2*>(a.q + t * a.H + v * 8) = encode8(u, s.of_u);
            if ((v & 15) == 0) static_cast<float*>(a.scales)[t * ((a.H + 127) / 128) + v / 16] = s.of_y;
        }
    } else if constexpr (FMT == kMX) {
        // largest pattern of the block's 4 lanes: from infinity's on the block has no codes
        const uint32_t top = dpp_umax<0x4E>(dpp_umax<0xB1>(__float_as_uint(amax8(y))));
        uint2 pk;
        int X = mx_encode8<false>(y, pk);
        if (top >= 0x7f800000u) {
            X = 128;
            pk = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
        }
        if (in) {
            *reinterpret_cast<uint2*>(a.q + t * a.H + v * 8) = pk;
            if ((v & 3) == 0) static_cast<uint8_t*>(a.scales)[t * (a.H / 32) + v / 4] = (uint8_t)(X + 127);
        }
    }
}

// A row's sum of squares and, for the rowwise format, its largest |u|, over the workgroup.
template <int NT, bool MAX>
__device__ __forceinline__ void row_sums(float& sum, uint32_t& top, float* s_sum, uint32_t* s_top) {
    sum = wave_sum(sum);
    if constexpr (MAX) top = wave_umax(top);
    if constexpr (NT > kWave) {
        if ((threadIdx.x & (kWave - 1)) == 0) {
            s_sum[threadIdx.x / kWave] = sum;
            if constexpr (MAX) s_top[threadIdx.x / kWave] = top;
        }
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NT / kWave; ++i) {
            sum += s_sum[i];
            if constexpr (MAX) top = max(top, s_top[i]);
        }
    }
}

// A workgroup of NT threads per row, VPT vectors of 8 elements a thread.
template <int NT, int VPT, int FMT, bool S32, bool RES>
__global__ __launch_bounds__(NT) void rmsnorm_kernel(const NormArgs a) {
    __shared__ float s_sum[2][NT / kWave];
    __shared__ uint32_t s_max[2][NT / kWave];
    constexpr bool kX32 = S32 && !RES;
    const int64_t nv = a.H / 8;
    float w[VPT][8];
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
        const int64_t v = threadIdx.x + NT * c;
        if (v < nv) load_weight8(a, v, w[c]);
    }
    int turn = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        float h[VPT][8];
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
            const int64_t v = threadIdx.x + NT * c;
            if (v < nv) {
                load8<kX32>(row_at<kX32>(a.x, t * a.H), v, h[c]);
                if constexpr (RES) {
                    float r[8];
                    load8<S32>(row_at<S32>(a.res, t * a.H), v, r);
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[c][i] += r[i];
                    if constexpr (!S32) {  // what the stream keeps
                        unpack8(pack8_bf16(h[c]), h[c]);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) h[c][i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(h[c][i], h[c][i], sum);
        }
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
            const int64_t v = threadIdx.x + NT * c;
            if constexpr (RES)
                if (v < nv) store8<S32>(row_at<S32>(a.h, t * a.H), v, h[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[c][i] = v < nv ? h[c][i] * w[c][i] : 0.0f;
            if constexpr (FMT == kRowwise) top = max(top, __float_as_uint(amax8(h[c])));
        }
        row_sums<NT, FMT == kRowwise>(sum, top, s_sum[turn], s_max[turn]);
        const float r = inverse_rms(sum, a.H, a.eps);
        Scale scale{};
        if constexpr (FMT == kRowwise) {
            scale = scale_of(__uint_as_float(top), r);
            if (threadIdx.x == 0) static_cast<float*>(a.scales)[t] = scale.of_y;
        }
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
            const int64_t v = threadIdx.x + NT * c;
            put8<FMT>(a, t, v, v < nv, h[c], r, scale);
        }
    }
}

// Rows longer than a workgroup's registers hold: the row is read again for each pass.
template <int NT, int FMT, bool S32, bool RES>
__global__ __launch_bounds__(NT) void rmsnorm_long_kernel(const NormArgs a) {
    __shared__ float s_sum[2][NT / kWave];
    __shared__ uint32_t s_max[2][NT / kWave];
    constexpr bool kX32 = S32 && !RES;
    const int64_t nv = a.H / 8, nv_up = (nv + NT - 1) / NT * NT;
    int turn = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        float sum = 0.0f;
        uint32_t top = 0;
        for (int64_t v = threadIdx.x; v < nv; v += NT) {
            float h[8], w[8];
            load8<kX32>(row_at<kX32>(a.x, t * a.H), v, h);
            if constexpr (RES) {
                float r[8];
                load8<S32>(row_at<S32>(a.res, t * a.H), v, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] += r[i];
                if constexpr (!S32) unpack8(pack8_bf16(h), h);
                store8<S32>(row_at<S32>(a.h, t * a.H), v, h);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(h[i], h[i], sum);
            if constexpr (FMT == kRowwise) {
                load_weight8(a, v, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] *= w[i];
                top = max(top, __float_as_uint(amax8(h)));
            }
        }
        row_sums<NT, FMT == kRowwise>(sum, top, s_sum[turn], s_max[turn]);
        const float r = inverse_rms(sum, a.H, a.eps);
        Scale scale{};
        if constexpr (FMT == kRowwise) {
            scale = scale_of(__uint_as_float(top), r);
            if (threadIdx.x == 0) static_cast<float*>(a.scales)[t] = scale.of_y;
        }
        // a thread reads back the vectors of h that it wrote itself
        for (int64_t v = threadIdx.x; v < nv_up; v += NT) {
            float u[8], w[8];
            if (v < nv) {
                load8<S32>(row_at<S32>(RES ? static_cast<const void*>(a.h) : a.x, t * a.H), v, u);
                load_weight8(a, v, w);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = v < nv ? u[i] * w[i] : 0.0f;
            put8<FMT>(a, t, v, v < nv, u, r, scale);
        }
    }
}

// ---------------------------------------------------------------------------
// The gradient.  One pass over the row: both of its sums, sum h^2 and sum g h, come
// from the registers that the outputs are made from, so the forward keeps no statistic.
// A workgroup adds up dy h r of its rows, its partial sum goes to a row of the workspace.
struct NormGradArgs {
    NormArgs n;  // x: dy, res: dh, h: the stream, y: dx_bf16, q: dx
    float* ws;
    int parts;   // rows of ws
};

template <int NT, int VPT, bool S32>
__global__ __launch_bounds__(NT) void rmsnorm_backward_kernel(const NormGradArgs ga) {
    const NormArgs& a = ga.n;
    __shared__ float s_sum[2][2][NT / kWave];
    const int64_t nv = a.H / 8;
    float w[VPT][8], dw[VPT][8];
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
        const int64_t v = threadIdx.x + NT * c;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[c][i] = dw[c][i] = 0.0f;
        if (v < nv) load_weight8(a, v, w[c]);
    }
    int turn = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        float h[VPT][8], d[VPT][8];
        float sum = 0.0f, dot = 0.0f;
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
            const int64_t v = threadIdx.x + NT * c;
            if (v < nv) {
                load8<S32>(row_at<S32>(static_cast<const void*>(a.h), t * a.H), v, h[c]);
                load8<false>(row_at<false>(a.x, t * a.H), v, d[c]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) h[c][i] = d[c][i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum = fmaf(h[c][i], h[c][i], sum);
                dot = fmaf(d[c][i] * w[c][i], h[c][i], dot);
            }
        }
        sum = wave_sum(sum);
        dot = wave_sum(dot);
        if constexpr (NT > kWave) {
            if ((threadIdx.x & (kWave - 1)) == 0) {
                s_sum[turn][0][threadIdx.x / kWave] = sum;
                s_sum[turn][1][threadIdx.x / kWave] = dot;
            }
            __syncthreads();
            sum = dot = 0.0f;
#pragma unroll
            for (int i = 0; i < NT / kWave; ++i) {
                sum += s_sum[turn][0][i];
                dot += s_sum[turn][1][i];
            }
        }
        const float r = inverse_rms(sum, a.H, a.eps);
        const float back = r * r * (dot * r / (float)a.H);  // of h
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
            const int64_t v = threadIdx.x + NT * c;
            if (v >= nv) continue;
            float dx[8];
            if (a.res) load8<S32>(row_at<S32>(a.res, t * a.H), v, dx);
            else
#pragma unroll
                for (int i = 0; i < 8; ++i) dx[i] = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dx[i] += r * (d[c][i] * w[c][i]) - h[c][i] * back;
                dw[c][i] = fmaf(d[c][i], h[c][i] * r, dw[c][i]);
            }
            if (a.q) store8<S32>(row_at<S32>(static_cast<void*>(a.q), t * a.H), v, dx);
            if (a.y) store8<false>(a.y + t * a.H, v, dx);
        }
    }
    if (ga.ws) {
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
            const int64_t v = threadIdx.x + NT * c;
            if (v < nv) store8_ws(ga.ws + blockIdx.x * a.H, v, dw[c]);
        }
    }
}

// Rows longer than the registers hold: read twice; the workgroup's sums stay in the
// workspace, whose columns each belong to one thread.
template <int NT, bool S32>
__global__ __launch_bounds__(NT) void rmsnorm_backward_long_kernel(const NormGradArgs ga) {
    const NormArgs& a = ga.n;
    __shared__ float s_sum[2][2][NT / kWave];
    const int64_t nv = a.H / 8;
    int turn = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        float sum = 0.0f, dot = 0.0f, h[8], d[8], w[8];
        for (int64_t v = threadIdx.x; v < nv; v += NT) {
            load8<S32>(row_at<S32>(static_cast<const void*>(a.h), t * a.H), v, h);
            load8<false>(row_at<false>(a.x, t * a.H), v, d);
            load_weight8(a, v, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum = fmaf(h[i], h[i], sum);
                dot = fmaf(d[i] * w[i], h[i], dot);
            }
        }
        sum = block_sum<NT>(sum, s_sum[turn][0]);
        dot = block_sum<NT>(dot, s_sum[turn][1]);
        const float r = inverse_rms(sum, a.H, a.eps);
        const float back = r * r * (dot * r / (float)a.H);
        for (int64_t v = threadIdx.x; v < nv; v += NT) {
            float dx[8], dw[8];
            load8<S32>(row_at<S32>(static_cast<const void*>(a.h), t * a.H), v, h);
            load8<false>(row_at<false>(a.x, t * a.H), v, d);
            load_weight8(a, v, w);
            if (a.res) load8<S32>(row_at<S32>(a.res, t * a.H), v, dx);
            else
#pragma unroll
                for (int i = 0; i < 8; ++i) dx[i] = 0.0f;
            if (ga.ws) {
                if (t == blockIdx.x)
#pragma unroll
                    for (int i = 0; i < 8; ++i) dw[i] = 0.0f;
                else load8_ws(ga.ws + blockIdx.x * a.H, v, dw);
#pragma unroll
                for (int i = 0; i < 8; ++i) dw[i] = fmaf(d[i], h[i] * r, dw[i]);
                store8_ws(ga.ws + blockIdx.x * a.H, v, dw);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) dx[i] += r * (d[i] * w[i]) - h[i] * back;
            if (a.q) store8<S32>(row_at<S32>(static_cast<void*>(a.q), t * a.H), v, dx);
            if (a.y) store8<false>(a.y + t * a.H, v, dx);
        }
    }
}

// dweight: the workspace's rows added up, 64 columns a workgroup (and 64 more each round of the launch), 16 rows at
// a time.
constexpr int kParts = 16;
__global__ __launch_bounds__(kWave * kParts) void rmsnorm_dweight_kernel(const float* __restrict__ ws, int parts,
                                                                         int64_t H, float* __restrict__ dw) {
    __shared__ float s[kParts][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    for (int64_t first = (int64_t)blockIdx.x * kWave; first < H; first += (int64_t)gridDim.x * kWave) {
        const int64_t col = first + lane;
        float v = 0.0f;
        if (col < H)
            for (int p = wave; p < parts; p += kParts) v += ws[p * H + col];
        s[wave][lane] = v;
        __syncthreads();
        if (wave == 0 && col < H) {
            v = 0.0f;
#pragma unroll
            for (int i = 0; i < kParts; ++i) v += s[i][lane];
            dw[col] = v;
        }
        __syncthreads();  // s is written again for the next columns
    }
}

constexpr int kMaxRow = 1024 * 8 * 4;  // elements a workgroup's registers hold

template <int FMT, bool S32, bool RES>
hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
    auto go = [&](auto kernel, int nt) {
        hipLaunchKernelGGL(kernel, dim3(workgroups(a.T, nt)), dim3(nt), 0, stream, a);
        return hipGetLastError();
    };
    if (a.H <= 512) return go(rmsnorm_kernel<64, 1, FMT, S32, RES>, 64);
    if (a.H <= 2048) return go(rmsnorm_kernel<64, 4, FMT, S32, RES>, 64);
    if (a.H <= 4096) return go(rmsnorm_kernel<256, 2, FMT, S32, RES>, 256);
    if (a.H <= 8192) return go(rmsnorm_kernel<256, 4, FMT, S32, RES>, 256);
    if (a.H <= kMaxRow) return go(rmsnorm_kernel<1024, 4, FMT, S32, RES>, 1024);
    return go(rmsnorm_long_kernel<1024, FMT, S32, RES>, 1024);
}

template <int FMT>
hipError_t launch_norm_fmt(bool s32, const NormArgs& a, hipStream_t stream) {
    if (a.res) return s32 ? launch_norm<FMT, true, true>(a, stream) : launch_norm<FMT, false, true>(a, stream);
    return s32 ? launch_norm<FMT, true, false>(a, stream) : launch_norm<FMT, false, false>(a, stream);
}

}  // namespace

hipError_t launch_rmsnorm(int fmt, bool s32, const void* x, const void* res, bool w32, const void* w, float w_add,
                          float eps, int64_t T, int64_t H, void* h, void* y, void* q, void* scales,
                          hipStream_t stream) {
    const NormArgs a{x, res, w, w_add, eps, T, H, h, static_cast<uint16_t*>(y), static_cast<uint8_t*>(q), scales, w32};
    switch (fmt) {
        case kPlain: return launch_norm_fmt<kPlain>(s32, a, stream);
        case kRowwise: return launch_norm_fmt<kRowwise>(s32, a, stream);
        case kMX: return launch_norm_fmt<kMX>(s32, a, stream);
        default: return launch_norm_fmt<kBlock>(s32, a, stream);
    }
}

int64_t rmsnorm_workspace_rows(int64_t T, int64_t) { return T < 512 ? T : 512; }

hipError_t launch_rmsnorm_backward(bool s32, const void* dy, const void* h, bool w32, const void* w, float w_add,
                                   float eps, const void* dh, int64_t T, int64_t H, void* dx, void* dx_bf16,
                                   float* dw, float* ws, hipStream_t stream) {
    const int parts = (int)rmsnorm_workspace_rows(T, H);
    if (T > 0) {
        const NormGradArgs a{{dy, dh, w, w_add, eps, T, H, const_cast<void*>(h), static_cast<uint16_t*>(dx_bf16),
                              static_cast<uint8_t*>(dx), nullptr, w32},
                             dw ? ws : nullptr, parts};
        auto go = [&](auto kernel, int nt) {
            hipLaunchKernelGGL(kernel, dim3((unsigned)parts), dim3(nt), 0, stream, a);
            return hipGetLastError();
        };
        auto pick = [&](auto f32) {
            constexpr bool S32 = decltype(f32)::value;
            if (H <= 512) return go(rmsnorm_backward_kernel<64, 1, S32>, 64);
            if (H <= 2048) return go(rmsnorm_backward_kernel<256, 1, S32>, 256);
            if (H <= 8192) return go(rmsnorm_backward_kernel<512, 2, S32>, 512);
            if (H <= 16384) return go(rmsnorm_backward_kernel<1024, 2, S32>, 1024);
            return go(rmsnorm_backward_long_kernel<1024, S32>, 1024);
        };
        const hipError_t e = s32 ? pick(std::true_type{}) : pick(std::false_type{});
        if (e != hipSuccess || !dw) return e;
    }
    hipLaunchKernelGGL(rmsnorm_dweight_kernel, dim3(workgroups((H + kWave - 1) / kWave, kWave * kParts)),
                       dim3(kWave * kParts), 0, stream, ws, T > 0 ? parts : 0, H, dw);
    return hipGetLastError();
}

}  // namespace mxg
