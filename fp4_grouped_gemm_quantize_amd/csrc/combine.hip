// combine.hip -- MoE combine after the down-projection, for gfx950: each token's
// output row is the router-weighted sum of the expert rows its slots were
// routed to.
//
// (grouped_matmul_rowwise_dynamic_scaled_fp8, Parameters: elementwise_lambda_fn
//  -- the optional output epilogue at (global_row, n) where this weighting and
//  the combine attach; NvMxf4f8Strategy, prepare_swiglu_operands(): the
//  EP-combine path; Struct_ep_dispatch_mxfp4: src_info, the source of each
//  dispatched row.)
//
// Design: a gather-sum per token instead of a scatter-add from the GEMM
// epilogue -- no atomics, no fp32 staging buffer, a fixed summation order
// (slot k = 0, 1, ...), so the result is deterministic.  One wave per token;
// each lane owns 8 consecutive outputs (16-byte loads of BF16 rows) per
// 512-wide chunk of H and keeps fp32 sums; the slot table is read by the
// lanes 64 entries at a time and broadcast with shuffles.  HBM traffic is the
// routed rows once plus the output once.
//
// Beside it: the rows' way into expert order (permute), whose gradient is the
// same gather-sum without weights, and the combine's own gradient.
#include "gemm_common.h"  // xcd_remap
#include "mxg_device.h"
#include "mxg_internal.h"

namespace mxg {

namespace {

constexpr int kThreads = 256;
constexpr int kWavesPerBlock = kThreads / kWave;
constexpr int kGather = 8;  // slot rows loaded together per lane

__global__ __launch_bounds__(kThreads) void combine_kernel(const uint16_t* __restrict__ y, int64_t T, int64_t H,
                                                           const int32_t* __restrict__ row_of_slot,
                                                           const float* __restrict__ wts, int64_t ntok, int top_k,
                                                           uint16_t* __restrict__ out) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t nunits = H / 8, step = (int64_t)gridDim.x * kWavesPerBlock;
    for (int64_t t = (int64_t)blockIdx.x * kWavesPerBlock + threadIdx.x / kWave; t < ntok; t += step) {  // wave-uniform
        const int32_t* slots = row_of_slot + t * top_k;
        const float* wt = wts + t * top_k;
        for (int64_t base = 0; base < nunits; base += kWave) {
            const int64_t u = base + lane;
            const bool on = u < nunits;
            float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            for (int k0 = 0; k0 < top_k; k0 += kWave) {
                const int kk = k0 + lane;
                int32_t r = -1;
                float wk = 0.0f;
                if (kk < top_k) {
                    r = slots[kk];
                    wk = wt[kk];
                }
                const int kn = top_k - k0 < kWave ? top_k - k0 : kWave;
                // slots in groups of kGather: all their row loads are issued
                // before any is accumulated (one load at a time left each wave
                // waiting out the memory latency per slot); the accumulation
                // order stays slot 0, 1, ...
                for (int j0 = 0; j0 < kn; j0 += kGather) {
                    uint4 v[kGather];
                    float wj[kGather];
                    bool use[kGather];
#pragma unroll
                    for (int q = 0; q < kGather; ++q) {
                        const int j = j0 + q < kn ? j0 + q : 0;  // uniform
                        const int32_t rj = __shfl(r, j, kWave);
                        wj[q] = __shfl(wk, j, kWave);
                        use[q] = j0 + q < kn && rj >= 0 && (int64_t)rj < T;  // wave-uniform: a dropped slot
                        v[q] = use[q] && on ? *reinterpret_cast<const uint4*>(y + (int64_t)rj * H + u * 8)
                                            : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int q = 0; q < kGather; ++q) {
                        if (!use[q] || !on) continue;
                        float f[8];
                        unpack8(v[q], f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[i] = fmaf(wj[q], f[i], acc[i]);
                    }
                }
            }
            if (on) {
                uint4 o;
                o.x = f32x2_to_bf16x2(acc[0], acc[1]);
                o.y = f32x2_to_bf16x2(acc[2], acc[3]);
                o.z = f32x2_to_bf16x2(acc[4], acc[5]);
                o.w = f32x2_to_bf16x2(acc[6], acc[7]);
                *reinterpret_cast<uint4*>(out + t * H + u * 8) = o;
            }
        }
    }
}

// The permutation, token-major: a wave reads one segment of a token's row once
// and stores it to the row of each of the token's slots (read once per slot the
// same rows would cross the fabric top_k times).  Bound by the stores, which are
// nontemporal: 8192 x 8 rows of 4096 122 us, 5.0 TB/s of which eight ninths are
// writes, and 106 where the last-level cache still holds the tokens.  (Ordinary
// stores 128; nontemporal loads 122 in either case; 2 and 8 KB a wave and slot
// instead of 4 no faster.)
constexpr int kSeg = 4;  // 16-byte vectors per lane per segment: 2048 elements a wave

__global__ __launch_bounds__(kThreads) void permute_kernel(const uint16_t* __restrict__ x, int64_t ntok, int64_t H,
                                                           int nseg, const int32_t* __restrict__ row_of_slot,
                                                           int top_k, uint16_t* __restrict__ rows, int64_t T) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t units = ntok * nseg, stride = (int64_t)gridDim.x * kWavesPerBlock, nunits = H / 8;
    for (int64_t u = (int64_t)blockIdx.x * kWavesPerBlock + threadIdx.x / kWave; u < units; u += stride) {
        const int64_t t = u / nseg, u0 = (u - t * nseg) * (kSeg * kWave) + lane;
        uint4 v[kSeg];
#pragma unroll
        for (int c = 0; c < kSeg; ++c)
            if (u0 + c * kWave < nunits) v[c] = *reinterpret_cast<const uint4*>(x + t * H + (u0 + c * kWave) * 8);
        for (int k0 = 0; k0 < top_k; k0 += kWave) {
            const int32_t mine = k0 + lane < top_k ? row_of_slot[t * top_k + k0 + lane] : -1;
            const int kn = top_k - k0 < kWave ? top_k - k0 : kWave;
            for (int k = 0; k < kn; ++k) {
                const int32_t r = __builtin_amdgcn_readlane(mine, k);
                if (r < 0 || (int64_t)r >= T) continue;  // a dropped slot (wave-uniform)
#pragma unroll
                for (int c = 0; c < kSeg; ++c)
                    if (u0 + c * kWave < nunits) store_stream16(rows + (int64_t)r * H + (u0 + c * kWave) * 8, v[c]);
            }
        }
    }
}

// The permutation's gradient: each token's row is the sum of its slots' rows,
// in slot order, in fp32.  A wave sums one 512-element piece of a token's row,
// so few tokens still fill the chip (4096 x 8 rows of 7168: 98 us, 5.4 TB/s).
__global__ __launch_bounds__(kThreads) void permute_backward_kernel(const uint16_t* __restrict__ drows, int64_t T,
                                                                    int64_t H, int nseg,
                                                                    const int32_t* __restrict__ row_of_slot,
                                                                    int64_t ntok, int top_k,
                                                                    uint16_t* __restrict__ dx) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t units = ntok * nseg, stride = (int64_t)gridDim.x * kWavesPerBlock;
    for (int64_t w = (int64_t)gemm::xcd_remap(blockIdx.x, gridDim.x) * kWavesPerBlock + threadIdx.x / kWave; w < units;
         w += stride) {
        const int64_t t = w / nseg;
        const int64_t u = (w - t * nseg) * kWave + lane;
        const bool on = u < H / 8;
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int k0 = 0; k0 < top_k; k0 += kWave) {
            const int32_t mine = k0 + lane < top_k ? row_of_slot[t * top_k + k0 + lane] : -1;
            const int kn = top_k - k0 < kWave ? top_k - k0 : kWave;
            for (int j0 = 0; j0 < kn; j0 += kGather) {
                uint4 v[kGather];
#pragma unroll
                for (int q = 0; q < kGather; ++q) {
                    const int32_t r = j0 + q < kn ? __builtin_amdgcn_readlane(mine, j0 + q) : -1;
                    const bool use = r >= 0 && (int64_t)r < T;
                    v[q] = use && on ? load_stream16(drows + (int64_t)r * H + u * 8) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int q = 0; q < kGather; ++q) {
                    float f[8];
                    unpack8(v[q], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] += f[i];
                }
            }
        }
        if (on) {
            uint4 o;
            o.x = f32x2_to_bf16x2(acc[0], acc[1]);
            o.y = f32x2_to_bf16x2(acc[2], acc[3]);
            o.z = f32x2_to_bf16x2(acc[4], acc[5]);
            o.w = f32x2_to_bf16x2(acc[6], acc[7]);
            *reinterpret_cast<uint4*>(dx + t * H + u * 8) = o;
        }
    }
}

// The combine's gradient: a workgroup per slot scales the token's gradient row
// into the slot's row and takes its dot product with the slot's y row (fp32 per
// lane, then over the wave, then over the waves: a fixed order).  Consecutive
// slots go to one XCD, so a token's row is fetched into one L2 for all of them.
// 4096 x 8 rows of 7168: 186 us, 5.4 TB/s (208 with ordinary stores).
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(
    const uint16_t* __restrict__ dout, const uint16_t* __restrict__ y, int64_t T, int64_t H,
    const int32_t* __restrict__ row_of_slot, const float* __restrict__ weights, int64_t nslots, int top_k,
    uint16_t* __restrict__ dy, float* __restrict__ dweights) {
    __shared__ float s_part[kWavesPerBlock];
    const int64_t nunits = H / 8;
    for (int64_t slot = gemm::xcd_remap(blockIdx.x, gridDim.x); slot < nslots; slot += gridDim.x) {
        const int32_t r = row_of_slot[slot];
        if (r < 0 || (int64_t)r >= T) {  // dropped (workgroup-uniform)
            if (threadIdx.x == 0) dweights[slot] = 0.0f;
            continue;
        }
        const float w = weights[slot];
        const uint16_t* d = dout + slot / top_k * H;
        const uint16_t* yr = y + (int64_t)r * H;
        uint16_t* dyr = dy + (int64_t)r * H;
        float dot = 0.0f;
#pragma unroll 4
        for (int64_t u = threadIdx.x; u < nunits; u += kThreads) {
            const uint4 dv = *reinterpret_cast<const uint4*>(d + u * 8);
            const uint4 yv = load_stream16(yr + u * 8);
            float a[8], b[8];
            unpack8(dv, a);
            unpack8(yv, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot = fmaf(a[i], b[i], dot);
            uint4 o;
            o.x = f32x2_to_bf16x2(w * a[0], w * a[1]);
            o.y = f32x2_to_bf16x2(w * a[2], w * a[3]);
            o.z = f32x2_to_bf16x2(w * a[4], w * a[5]);
            o.w = f32x2_to_bf16x2(w * a[6], w * a[7]);
            store_stream16(dyr + u * 8, o);
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) dot += __shfl_xor(dot, o, kWave);
        if ((threadIdx.x & (kWave - 1)) == 0) s_part[threadIdx.x / kWave] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
            float sum = s_part[0];
#pragma unroll
            for (int i = 1; i < kWavesPerBlock; ++i) sum += s_part[i];
            dweights[slot] = sum;
        }
        __syncthreads();  // s_part is written again for the next slot
    }
}

// A launch holds fewer than 2^32 threads; past this many workgroups they loop.
unsigned grid_of(int64_t blocks) { return (unsigned)(blocks < (1 << 20) ? blocks : 1 << 20); }

}  // namespace

hipError_t launch_permute(const void* x, int64_t ntok, int64_t H, const int32_t* row_of_slot, int top_k, void* rows,
                          int64_t T, hipStream_t stream) {
    const int64_t nseg = (H / 8 + kSeg * kWave - 1) / (kSeg * kWave);
    const int64_t blocks = (ntok * nseg + kWavesPerBlock - 1) / kWavesPerBlock;
    hipLaunchKernelGGL(permute_kernel, dim3(grid_of(blocks)), dim3(kThreads), 0, stream,
                       static_cast<const uint16_t*>(x), ntok, H, (int)nseg, row_of_slot, top_k,
                       static_cast<uint16_t*>(rows), T);
    return hipGetLastError();
}

hipError_t launch_permute_backward(const void* drows, int64_t T, int64_t H, const int32_t* row_of_slot, int64_t ntok,
                                   int top_k, void* dx, hipStream_t stream) {
    const int64_t nseg = (H / 8 + kWave - 1) / kWave;
    const int64_t blocks = (ntok * nseg + kWavesPerBlock - 1) / kWavesPerBlock;
    hipLaunchKernelGGL(permute_backward_kernel, dim3(grid_of(blocks)), dim3(kThreads), 0, stream,
                       static_cast<const uint16_t*>(drows), T, H, (int)nseg, row_of_slot, ntok, top_k,
                       static_cast<uint16_t*>(dx));
    return hipGetLastError();
}

hipError_t launch_combine_backward(const void* dout, const void* y, int64_t T, int64_t H, const int32_t* row_of_slot,
                                   const float* weights, int64_t ntok, int top_k, void* dy, float* dweights,
                                   hipStream_t stream) {
    const int64_t nslots = ntok * top_k;  // at most INT32_MAX
    hipLaunchKernelGGL(combine_backward_kernel, dim3(grid_of(nslots)), dim3(kThreads), 0, stream,
                       static_cast<const uint16_t*>(dout), static_cast<const uint16_t*>(y), T, H, row_of_slot,
                       weights, nslots, top_k, static_cast<uint16_t*>(dy), dweights);
    return hipGetLastError();
}

hipError_t launch_combine(const void* y, int64_t T, int64_t H, const int32_t* row_of_slot, const float* weights,
                          int64_t ntok, int top_k, void* out, hipStream_t stream) {
    hipLaunchKernelGGL(combine_kernel, dim3(grid_of((ntok + kWavesPerBlock - 1) / kWavesPerBlock)), dim3(kThreads), 0,
                       stream, static_cast<const uint16_t*>(y), T, H, row_of_slot, weights, ntok, top_k,
                       static_cast<uint16_t*>(out));
    return hipGetLastError();
}

}  // namespace mxg
