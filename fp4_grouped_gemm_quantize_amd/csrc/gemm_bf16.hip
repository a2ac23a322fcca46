// gemm_bf16.hip -- ragged grouped product of BF16 operands with bias, activation and
// residual in its epilogue, the gradient of its rows through the activation before
// them, and the activation's gradient by itself, for gfx950.
#include "gemm_bf16.h"

namespace mxg {

using namespace bf16;

namespace {

constexpr int kTile = 64, kDepth = 32, kPitch = kDepth + 8, kThreads = 256;

// One 64 x 64 tile a workgroup: blockIdx.x the column tile, blockIdx.y the row tile
// among all groups' (found by a walk over the groups).
template <bool BACK>
__global__ __launch_bounds__(kThreads) void matmul_bf16_kernel(const Bf16Problem p) {
    __shared__ __attribute__((aligned(16))) uint16_t s_a[kTile * kPitch], s_b[kTile * kPitch];
    const int64_t cols = BACK ? p.K : p.N, depth = BACK ? p.N : p.K;
    int64_t left = blockIdx.y;
    int g = 0;
    GroupRange r{0, 0};
    for (; g < p.G; ++g) {
        r = rows_of(p.off, p.ids, g, p.T, p.E);
        const int64_t tiles = (r.hi - r.lo + kTile - 1) / kTile;
        if (left < tiles) break;
        left -= tiles;
    }
    if (g == p.G) return;
    const int e = expert_of(p.ids, g);
    const int64_t m0 = r.lo + left * kTile, n0 = (int64_t)blockIdx.x * kTile;
    const uint16_t* a = static_cast<const uint16_t*>(p.a);
    const uint16_t* b = static_cast<const uint16_t*>(p.b) + (int64_t)e * p.N * p.K;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid / 64, wm = wave / 2, wn = wave % 2, l16 = lane & 15,
              kg = lane >> 4;
    v4f acc[2][2];
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int64_t k0 = 0; k0 < depth; k0 += kDepth) {
        {
            const int row = tid / 4, piece = tid % 4;
            const int64_t k = k0 + piece * 8;
            uint4 v = make_uint4(0, 0, 0, 0), w = v;
            if (m0 + row < r.hi && k < depth) v = *reinterpret_cast<const uint4*>(a + (m0 + row) * depth + k);
            *reinterpret_cast<uint4*>(s_a + row * kPitch + piece * 8) = v;
            if constexpr (!BACK) {
                if (n0 + row < cols && k < depth) w = *reinterpret_cast<const uint4*>(b + (n0 + row) * depth + k);
                *reinterpret_cast<uint4*>(s_b + row * kPitch + piece * 8) = w;
            } else {
                const int kr = tid / 8, c8 = (tid % 8) * 8;
                if (k0 + kr < depth && n0 + c8 < cols)
                    w = *reinterpret_cast<const uint4*>(b + (k0 + kr) * cols + n0 + c8);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
                for (int i = 0; i < 8; ++i) s_b[(c8 + i) * kPitch + kr] = (uint16_t)(ww[i / 2] >> (16 * (i & 1)));
            }
        }
        __syncthreads();
        v8b fa[2], fb[2];
        for (int i = 0; i < 2; ++i) {
            fa[i] = *reinterpret_cast<const v8b*>(s_a + (wm * 32 + i * 16 + l16) * kPitch + kg * 8);
            fb[i] = *reinterpret_cast<const v8b*>(s_b + (wn * 32 + i * 16 + l16) * kPitch + kg * 8);
        }
        for (int i = 0; i < 2; ++i)
            for (int j = 0; j < 2; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[i], fa[j], acc[i][j], 0, 0, 0);
        __syncthreads();
    }
    with_act(p.act, [&](auto act) {
        for (int j = 0; j < 2; ++j) {
            const int64_t t = m0 + wm * 32 + j * 16 + l16;
            if (t >= r.hi) continue;
            for (int i = 0; i < 2; ++i) {
                const int64_t col = n0 + wn * 32 + i * 16 + kg * 4;
                if (col >= cols) continue;
                const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                if constexpr (BACK) finish4_backward<act()>(p, t, col, v);
                else finish4<act()>(p, e, t, col, v);
            }
        }
    });
}

template <bool BACK>
hipError_t launch(const Bf16Problem& p, hipStream_t stream) {
    const int64_t cols = BACK ? p.K : p.N;
    const dim3 grid((unsigned)((cols + kTile - 1) / kTile), (unsigned)(p.T / kTile + p.G));
    hipLaunchKernelGGL(matmul_bf16_kernel<BACK>, grid, dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// The activation's gradient by itself: 8 values of z a thread (swiglu: 4 pairs).
template <int ACT>
__global__ __launch_bounds__(256) void activation_backward_kernel(const void* dc, const void* z, void* dz,
                                                                  int64_t units) {
    for (int64_t u = blockIdx.x * 256LL + threadIdx.x; u < units; u += gridDim.x * 256LL) {
        float zv[8], out[8];
        load_n<8>(static_cast<const uint16_t*>(z) + u * 8, false, true, 8, zv);
        if constexpr (ACT == kSwiglu) {
            float d[4];
            load_n<4>(static_cast<const uint16_t*>(dc) + u * 4, false, true, 4, d);
            swiglu_grad4(zv, d, out);
        } else {
            load_n<8>(static_cast<const uint16_t*>(dc) + u * 8, false, true, 8, out);
#pragma unroll
            for (int i = 0; i < 8; ++i) out[i] *= derivative<ACT>(zv[i]);
        }
        store_n<8>(static_cast<uint16_t*>(dz) + u * 8, false, true, 8, out);
    }
}

}  // namespace

hipError_t launch_matmul_bf16(const Bf16Problem& p, hipStream_t stream) { return launch<false>(p, stream); }
hipError_t launch_matmul_bf16_backward(const Bf16Problem& p, hipStream_t stream) { return launch<true>(p, stream); }

hipError_t launch_activation_backward(int act, const void* dc, const void* z, void* dz, int64_t T, int64_t N,
                                      hipStream_t stream) {
    const int64_t units = T * N / (act == kSwiglu ? 4 : 8), blocks = (units + 255) / 256;
    const dim3 grid((unsigned)(blocks < (1 << 24) ? blocks : (1 << 24)));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, dc, z, dz, units);
        return hipGetLastError();
    };
    switch (act) {
        case kRelu: return go(activation_backward_kernel<kRelu>);
        case kGelu: return go(activation_backward_kernel<kGelu>);
        case kSilu: return go(activation_backward_kernel<kSilu>);
        default: return go(activation_backward_kernel<kSwiglu>);
    }
}

}  // namespace mxg
