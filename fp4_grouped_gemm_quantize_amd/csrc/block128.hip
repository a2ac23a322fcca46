// block128.hip -- FP8 e4m3 with an fp32 scale per 128-element block: the
// quantisers of activations (1 x 128) and weights (128 x 128, plain and
// transposed), and SwiGLU with that requant and its gradient, for gfx950.
//
// (NvMxf4f8Strategy, grouped_quantize() and fused_silu_quantize(), in a block
//  format the pages do not have: scale = amax / 448, code = e4m3(x / scale).)
//
// All are HBM-bound streams read once and written once.  16 lanes x 8 elements
// form a 1 x 128 block, so a wave's 16-byte loads stay contiguous and the block
// maximum is four register exchanges.  Every wave takes one unit of work and
// ends: persistent waves that load the next unit while they encode the current
// one were slower at every grid size (SwiGLU gradient of 32768 x 2048, inputs in
// the last-level cache: 179 us with 8 resident workgroups a CU, 156 with 4, 161
// with 64, 147 so).  Which streams carry the nontemporal hint is by measurement
// on inputs that no cache holds, and stated at each kernel; the times there are
// of such inputs too.
#include "mxg_device.h"
#include "mxg_internal.h"

namespace mxg {

namespace {

constexpr int kThreads = 256;
constexpr int kWavesPerBlock = kThreads / kWave;
constexpr int kChunk = kWave * 8;  // elements per wave-wide load
constexpr int kBlk = 128;

// Largest magnitude of 8 values, as the integer order of the magnitudes has it:
// a NaN's pattern lies above infinity's, so a block with a NaN gets a NaN scale
// (a floating-point maximum would drop it).
__device__ __forceinline__ float amax8(const float* f) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(f[i]) & 0x7fffffffu);
    return __uint_as_float(a);
}
// The same maximum over 8 (16) neighbouring lanes: lane ^ 1, lane ^ 2, then the
// mirrors within 8 (and 16) lanes.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float amax_of8(float v) {
    return __uint_as_float(dpp_umax<0x141>(dpp_umax<0x4E>(dpp_umax<0xB1>(__float_as_uint(v)))));
}
__device__ __forceinline__ float amax_of16(float v) {
    return __uint_as_float(dpp_umax<0x140>(__float_as_uint(amax_of8(v))));
}

// Codes of 8 values under their block's scale: e4m3(x / scale), the code of the
// quotient that IEEE binary32 division gives.  One division gives the scale's
// reciprocal r; each quotient is then x r corrected by its exact remainder,
// q + (x - q scale) r (Markstein), three operations instead of a division's ten.
// Scales below 2^-60 are lifted by 2^64 with their values, an exact step, so that
// neither the reciprocal overflows nor the remainder underflows.  (Checked on the
// CPU: the codes equal those of the division for every bf16 maximum and every bf16
// value up to it, and for 480 M fp32 pairs, half of them next to a code's border;
// only quotients far below the smallest code differ from the division's.)  Under an
// infinite scale r is 0 and the remainder is taken with the largest finite number
// instead, since 0 times infinity would make the quotient of a finite value, 0, a
// NaN; an infinity over it stays one.  The clamp matters only where the scale is a
// subnormal that rounded down.
__device__ __forceinline__ uint2 encode8(const float* x, float scale) {
    float f[8];
    if (scale == 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = x[i] * 0.0f;
    } else {
        const float lift = scale < 0x1p-60f ? 0x1p64f : 1.0f;
        const float lifted = scale * lift, r = 1.0f / lifted, s = fminf(lifted, 0x1.fffffep127f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float xi = x[i] * lift, q = xi * r;
            const float v = copysignf(fmaf(fmaf(-q, s, xi), r, q), q);  // (a remainder of 0 would turn -0 into 0)
            f[i] = v > 448.0f ? 448.0f : v < -448.0f ? -448.0f : v;  // keeps a NaN
        }
    }
    return pack8_e4m3(f);
}

// 8 bytes with the nontemporal hint.
__device__ __forceinline__ void store_stream8(void* p, const uint2& v) {
    typedef unsigned u2v __attribute__((ext_vector_type(2)));
    u2v t;
    t.x = v.x;
    t.y = v.y;
    __builtin_nontemporal_store(t, static_cast<u2v*>(p));
}

__device__ __forceinline__ void load_offsets(uint32_t* s_off, const uint32_t* off, int G) {
    for (int i = threadIdx.x; i <= G; i += blockDim.x) s_off[i] = off[i];
    __syncthreads();
}

// ---------------------------------------------------------------------------
// Rows of bf16.  A unit is a row's segment of kNC 512-element chunks; the codes are
// nontemporal (8192 x 4096 scattered to 65536 rows: 68 us, 5.0 TB/s; 72 with ordinary
// stores), the loads are not: 55 us where the last-level cache still holds the rows,
// 68 with nontemporal loads in either case.  Row-major, 65536 x 4096 of 128 groups: 154
// to 160 us, 5.1 to 5.3 TB/s, with nontemporal loads the same (8192 x 4096: 21.4 and
// 20.9, from the cache 19.7 and 20.6), ordinary stores 1 to 7 % more.  Every workgroup
// copies the offsets and every wave looks through them: 1024 groups take 207.
// SCATTER: unit rows are tokens, encoded once and stored to the rows of the
// token's slots (top_k <= 64: lane k holds slot k).
constexpr int kNC = 2;

template <bool SCATTER>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(const uint16_t* __restrict__ x, int64_t nrow,
                                                                 const int32_t* __restrict__ ros, int top_k,
                                                                 uint8_t* __restrict__ q, float* __restrict__ scales,
                                                                 const uint32_t* __restrict__ off, int G, int64_t T,
                                                                 int64_t K, int nseg) {
    __shared__ uint32_t s_off[kMaxGroups + 1];
    load_offsets(s_off, off, G);
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t units = nrow * nseg, step = (int64_t)gridDim.x * kWavesPerBlock;
    const int64_t nblk = (K + kBlk - 1) / kBlk;
    auto load = [&](int64_t u, uint4 (&v)[kNC]) {
        const int64_t r = u / nseg;
        const int64_t e0 = (u - r * nseg) * (kNC * kChunk) + lane * 8;
#pragma unroll
        for (int c = 0; c < kNC; ++c)
            v[c] = e0 + c * kChunk < K ? *reinterpret_cast<const uint4*>(x + r * K + e0 + c * kChunk)
                                       : make_uint4(0, 0, 0, 0);
    };
    uint4 v[kNC];
    for (int64_t u = (int64_t)blockIdx.x * kWavesPerBlock + wave; u < units; u += step) {
        load(u, v);
        const int64_t r = u / nseg;
        const int64_t e0 = (u - r * nseg) * (kNC * kChunk) + lane * 8;
        int32_t mine = -1;
        if constexpr (SCATTER) mine = lane < top_k ? ros[r * top_k + lane] : -1;
        const bool taken = SCATTER || wave_row_covered(s_off, G, T, r);
        if (taken) {
            uint2 pk[kNC];
            float sc[kNC];
#pragma unroll
            for (int c = 0; c < kNC; ++c) {
                float f[8];
                unpack8(v[c], f);
                sc[c] = amax_of16(amax8(f)) / 448.0f;  // IEEE binary32 division
                pk[c] = encode8(f, sc[c]);
            }
            auto store = [&](int64_t t) {
#pragma unroll
                for (int c = 0; c < kNC; ++c) {
                    const int64_t e = e0 + c * kChunk;
                    if (e >= K) continue;
                    store_stream8(q + t * K + e, pk[c]);
                    if ((lane & 15) == 0) scales[t * nblk + e / kBlk] = sc[c];
                }
            };
            if constexpr (SCATTER) {
                for (int k = 0; k < top_k; ++k) {
                    const int32_t t = __builtin_amdgcn_readlane(mine, k);
                    if (t >= 0 && (int64_t)t < T && wave_row_covered(s_off, G, T, t)) store(t);
                }
            } else {
                store(r);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Weights: a workgroup per 128 x 128 tile, 16 lanes a row (128 elements), the
// tile held in registers between the maximum and the encoding.  The transposed
// codes go through LDS as words of four columns; a thread gathers four columns
// of 16 rows and turns 4 x 4 byte blocks round with byte permutes, so both
// layouts leave in 16-byte (plain: 8-byte) pieces of whole 128-byte lines, both
// nontemporal: 8 x 4096 x 7168 in both layouts 178 us (5.3 TB/s), 185 with either
// or neither so.
constexpr int kPitch = 33;  // words a tile row in LDS (32 and one against bank conflicts)

__global__ __launch_bounds__(kThreads) void quantize_weights_kernel(const uint16_t* __restrict__ w, int64_t E,
                                                                    int64_t N, int64_t K, uint8_t* __restrict__ q,
                                                                    float* __restrict__ scales,
                                                                    uint8_t* __restrict__ qt,
                                                                    float* __restrict__ scales_t) {
    __shared__ uint32_t s_tile[kBlk * kPitch];
    __shared__ uint32_t s_max[kWavesPerBlock];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int64_t nn = (N + kBlk - 1) / kBlk, nk = (K + kBlk - 1) / kBlk, tiles = E * nn * nk;
    const int r0 = tid / 16, c8 = (tid % 16) * 8;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t kb = tile % nk, en = tile / nk, nb = en % nn, e = en / nn;
        const int64_t n0 = nb * kBlk, k0 = kb * kBlk;
        const bool in_k = k0 + c8 < K;
        uint4 v[8];
        uint32_t a = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t n = n0 + r0 + 16 * i;
            v[i] = in_k && n < N ? load_stream16(w + (e * N + n) * K + k0 + c8) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float f[8];
            unpack8(v[i], f);
            a = max(a, __float_as_uint(amax8(f)));
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) a = max(a, (uint32_t)__shfl_xor((int)a, o, kWave));
        if (lane == 0) s_max[wave] = a;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWavesPerBlock; ++i) a = max(a, s_max[i]);
        const float sc = __uint_as_float(a) / 448.0f;
        if (tid == 0) {
            scales[(e * nn + nb) * nk + kb] = sc;
            if (qt) scales_t[(e * nk + kb) * nn + nb] = sc;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + 16 * i;
            const int64_t n = n0 + r;
            float f[8];
            unpack8(v[i], f);
            const uint2 p = encode8(f, sc);
            if (in_k && n < N) store_stream8(q + (e * N + n) * K + k0 + c8, p);
            if (qt) {
                s_tile[r * kPitch + c8 / 4] = p.x;
                s_tile[r * kPitch + c8 / 4 + 1] = p.y;
            }
        }
        __syncthreads();
        if (qt) {
            const int kw = tid / 8, nr = (tid % 8) * 16;  // columns 4 kw .. + 3, rows nr .. + 15
            uint32_t o[4][4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t a0 = s_tile[(nr + 4 * b) * kPitch + kw], a1 = s_tile[(nr + 4 * b + 1) * kPitch + kw];
                uint32_t a2 = s_tile[(nr + 4 * b + 2) * kPitch + kw], a3 = s_tile[(nr + 4 * b + 3) * kPitch + kw];
                const uint32_t lo01 = __builtin_amdgcn_perm(a1, a0, 0x05010400u);  // a0.0 a1.0 a0.1 a1.1
                const uint32_t hi01 = __builtin_amdgcn_perm(a1, a0, 0x07030602u);
                const uint32_t lo23 = __builtin_amdgcn_perm(a3, a2, 0x05010400u);
                const uint32_t hi23 = __builtin_amdgcn_perm(a3, a2, 0x07030602u);
                o[0][b] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
                o[1][b] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
                o[2][b] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
                o[3][b] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int64_t k = k0 + 4 * kw + c;
                if (k < K && n0 + nr < N)  // N is a multiple of 32: the 16 rows are all in or all out
                    store_stream16(qt + (e * K + k) * N + n0 + nr, make_uint4(o[c][0], o[c][1], o[c][2], o[c][3]));
            }
        }
        // the next tile writes s_max before its first barrier and s_tile after it
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// SwiGLU.  silu(g) = g s with s = 1 / (1 + e^-g), by the hardware's exp2 and
// reciprocal (one ulp each, and the rounding of g log2 e: a relative 2^-23 times
// |g|, far below the codes' 2^-4 and within the scales' own rounding for the |g|
// whose activation is not negligible; a sigmoid below fp32's normal range, from g =
// -87.3 on, may be 0, which leaves out less than |g u| 2^-125).  Against 64 bits 218 of 33 M codes of the
// gradient differ, by the rounding of scale and quotient that the format fixes: a
// sigmoid of half the error and exact BF16 products leave 222 and cost 5 %.
__device__ __forceinline__ float fast_sigmoid(float g) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896340736f));
}

// A unit is 512 outputs of a row: a lane's 8 outputs are 16 of h (two 16-byte
// loads), 16 lanes a block; the codes are nontemporal (32768 x 2048: 67 us, 5.0
// TB/s; 72 with ordinary stores, 69 with nontemporal loads).
__global__ __launch_bounds__(kThreads) void silu_quantize_kernel(const uint16_t* __restrict__ h,
                                                                 uint8_t* __restrict__ q, float* __restrict__ scales,
                                                                 const uint32_t* __restrict__ off, int G, int64_t T,
                                                                 int64_t I, int nseg) {
    __shared__ uint32_t s_off[kMaxGroups + 1];
    load_offsets(s_off, off, G);
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t units = T * nseg, step = (int64_t)gridDim.x * kWavesPerBlock, nblk = (I + kBlk - 1) / kBlk;
    auto load = [&](int64_t u, uint4 (&v)[2]) {
        const int64_t r = u / nseg, j = (u - r * nseg) * kChunk + lane * 8;
        const bool in = j < I;
        const uint16_t* p = h + r * 2 * I + 2 * j;
#pragma unroll
        for (int c = 0; c < 2; ++c) v[c] = in ? *reinterpret_cast<const uint4*>(p + 8 * c) : make_uint4(0, 0, 0, 0);
    };
    uint4 v[2];
    for (int64_t u = (int64_t)blockIdx.x * kWavesPerBlock + wave; u < units; u += step) {
        load(u, v);
        const int64_t r = u / nseg, j = (u - r * nseg) * kChunk + lane * 8;
        if (wave_row_covered(s_off, G, T, r)) {
            float gu[16], y[8];
            unpack8(v[0], gu);
            unpack8(v[1], gu + 8);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = gu[2 * i] * fast_sigmoid(gu[2 * i]) * gu[2 * i + 1];
            const float sc = amax_of16(amax8(y)) / 448.0f;
            const uint2 p = encode8(y, sc);
            if (j < I) {
                store_stream8(q + r * I + j, p);
                if ((lane & 15) == 0) scales[r * nblk + j / kBlk] = sc;
            }
        }
    }
}

// The gradient: a lane's 8 outputs give 16 elements of dh, so 8 lanes are a
// block of dh.  No stream is nontemporal (32768 x 2048, dh kept and quantised:
// 144 us, 5.6 TB/s; 149 with the loads so, 157 with dh too, 166 with all).  dh may
// be h itself: a lane has read its elements before it writes them, and no other
// lane reads them.
template <bool KEEP, bool QUANT>
__global__ __launch_bounds__(kThreads) void silu_backward_kernel(const uint16_t* h, const uint16_t* __restrict__ dy,
                                                                 uint16_t* dh, uint8_t* __restrict__ q,
                                                                 float* __restrict__ scales,
                                                                 const uint32_t* __restrict__ off, int G, int64_t T,
                                                                 int64_t I, int nseg) {
    __shared__ uint32_t s_off[kMaxGroups + 1];
    load_offsets(s_off, off, G);
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t units = T * nseg, step = (int64_t)gridDim.x * kWavesPerBlock, nblk = (2 * I + kBlk - 1) / kBlk;
    auto load = [&](int64_t u, uint4 (&v)[3]) {
        const int64_t r = u / nseg, j = (u - r * nseg) * kChunk + lane * 8;
        const bool in = j < I;
        const uint16_t* p = h + r * 2 * I + 2 * j;
        v[0] = in ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
        v[1] = in ? *reinterpret_cast<const uint4*>(p + 8) : make_uint4(0, 0, 0, 0);
        v[2] = in ? *reinterpret_cast<const uint4*>(dy + r * I + j) : make_uint4(0, 0, 0, 0);
    };
    uint4 v[3];
    for (int64_t u = (int64_t)blockIdx.x * kWavesPerBlock + wave; u < units; u += step) {
        load(u, v);
        const int64_t r = u / nseg, j = (u - r * nseg) * kChunk + lane * 8;
        if (wave_row_covered(s_off, G, T, r)) {
            float gu[16], d[8], o[16];
            unpack8(v[0], gu);
            unpack8(v[1], gu + 8);
            unpack8(v[2], d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float g = gu[2 * i], s = fast_sigmoid(g);
                const float ds = d[i] * s;
                o[2 * i] = ds * gu[2 * i + 1] * fmaf(g, 1.0f - s, 1.0f);
                o[2 * i + 1] = ds * g;
            }
            if constexpr (KEEP) {
                if (j < I) {
                    uint4 w[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        w[c].x = f32x2_to_bf16x2(o[8 * c], o[8 * c + 1]);
                        w[c].y = f32x2_to_bf16x2(o[8 * c + 2], o[8 * c + 3]);
                        w[c].z = f32x2_to_bf16x2(o[8 * c + 4], o[8 * c + 5]);
                        w[c].w = f32x2_to_bf16x2(o[8 * c + 6], o[8 * c + 7]);
                        *reinterpret_cast<uint4*>(dh + r * 2 * I + 2 * j + 8 * c) = w[c];
                    }
                }
            }
            if constexpr (QUANT) {
                const uint32_t top = max(__float_as_uint(amax8(o)), __float_as_uint(amax8(o + 8)));
                const float sc = amax_of8(__uint_as_float(top)) / 448.0f;
                const uint2 p0 = encode8(o, sc), p1 = encode8(o + 8, sc);
                if (j < I) {
                    *reinterpret_cast<uint4*>(q + r * 2 * I + 2 * j) = make_uint4(p0.x, p0.y, p1.x, p1.y);
                    if ((lane & 7) == 0) scales[r * nblk + 2 * j / kBlk] = sc;
                }
            }
        }
    }
}

// A wave per unit; a launch holds fewer than 2^32 threads, past this many workgroups they loop.
unsigned grid_of(int64_t units) {
    const int64_t blocks = (units + kWavesPerBlock - 1) / kWavesPerBlock;
    return (unsigned)(blocks < (1 << 20) ? blocks : 1 << 20);
}

}  // namespace

hipError_t launch_quantize_block128(const void* x, int64_t ntok, const int32_t* row_of_slot, int top_k, void* q,
                                    float* scales, const uint32_t* off, int G, int64_t T, int64_t K,
                                    hipStream_t stream) {
    const int64_t nseg = (K + kNC * kChunk - 1) / (kNC * kChunk);
    const dim3 grid(grid_of(ntok * nseg));
    if (row_of_slot)
        hipLaunchKernelGGL(quantize_rows_kernel<true>, grid, dim3(kThreads), 0, stream,
                           static_cast<const uint16_t*>(x), ntok, row_of_slot, top_k, static_cast<uint8_t*>(q),
                           scales, off, G, T, K, (int)nseg);
    else
        hipLaunchKernelGGL(quantize_rows_kernel<false>, grid, dim3(kThreads), 0, stream,
                           static_cast<const uint16_t*>(x), ntok, row_of_slot, top_k, static_cast<uint8_t*>(q),
                           scales, off, G, T, K, (int)nseg);
    return hipGetLastError();
}

hipError_t launch_quantize_weights_block128(const void* w, int64_t E, int64_t N, int64_t K, void* q, float* scales,
                                            void* q_t, float* scales_t, hipStream_t stream) {
    const int64_t tiles = E * ((N + kBlk - 1) / kBlk) * ((K + kBlk - 1) / kBlk);
    const unsigned grid = (unsigned)(tiles < (1 << 20) ? tiles : 1 << 20);
    hipLaunchKernelGGL(quantize_weights_kernel, dim3(grid), dim3(kThreads), 0, stream,
                       static_cast<const uint16_t*>(w), E, N, K, static_cast<uint8_t*>(q), scales,
                       static_cast<uint8_t*>(q_t), scales_t);
    return hipGetLastError();
}

hipError_t launch_silu_quantize_block128(const void* h, void* yq, float* ys, const uint32_t* off, int G, int64_t T,
                                         int64_t I, hipStream_t stream) {
    const int64_t nseg = (I + kChunk - 1) / kChunk;
    hipLaunchKernelGGL(silu_quantize_kernel, dim3(grid_of(T * nseg)), dim3(kThreads), 0, stream,
                       static_cast<const uint16_t*>(h), static_cast<uint8_t*>(yq), ys, off, G, T, I, (int)nseg);
    return hipGetLastError();
}

hipError_t launch_silu_backward_block128(const void* h, const void* dy, void* dh, void* dh_q, float* dh_scales,
                                         const uint32_t* off, int G, int64_t T, int64_t I, hipStream_t stream) {
    const int64_t nseg = (I + kChunk - 1) / kChunk;
    const dim3 grid(grid_of(T * nseg));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, static_cast<const uint16_t*>(h),
                           static_cast<const uint16_t*>(dy), static_cast<uint16_t*>(dh), static_cast<uint8_t*>(dh_q),
                           dh_scales, off, G, T, I, (int)nseg);
        return hipGetLastError();
    };
    if (dh && dh_q) return go(silu_backward_kernel<true, true>);
    return dh ? go(silu_backward_kernel<true, false>) : go(silu_backward_kernel<false, true>);
}

}  // namespace mxg
