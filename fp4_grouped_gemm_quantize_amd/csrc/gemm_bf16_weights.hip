// gemm_bf16_weights.hip -- the gradient of the experts' weights and biases: for each
// expert the product of its rows' gradients, transposed, with its rows, for gfx950.
#include "gemm_bf16.h"

namespace mxg {

using namespace bf16;

namespace {

constexpr int kTile = 64, kDepth = 32, kPitch = kDepth + 8, kThreads = 256;

struct WeightsArgs {
    const uint16_t* dc;
    const uint16_t* a;
    void* dw;
    float* dbias;
    const uint32_t* off;
    const int32_t* ids;
    int G, E;
    int64_t T, N, K;
    bool dw32, accumulate;
};

// One 64 x 64 tile of one expert's dw a workgroup.
__global__ __launch_bounds__(kThreads) void weights_kernel(const WeightsArgs p) {
    __shared__ __attribute__((aligned(16))) uint16_t s_n[kTile * kPitch], s_k[kTile * kPitch];
    const int64_t nk = (p.K + kTile - 1) / kTile;
    const int64_t n0 = blockIdx.x / nk * kTile, k0 = blockIdx.x % nk * kTile;
    const int e = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid / 64, wm = wave / 2, wn = wave % 2, l16 = lane & 15,
              kg = lane >> 4;
    v4f acc[2][2];
    float bsum = 0.0f;
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int g = 0; g < p.G; ++g) {
        if (expert_of(p.ids, g) != e) continue;
        const GroupRange r = rows_of(p.off, p.ids, g, p.T, p.E);
        for (int64_t t0 = r.lo; t0 < r.hi; t0 += kDepth) {
            const int tr = tid / 8, c8 = (tid % 8) * 8;
            uint4 v = make_uint4(0, 0, 0, 0), w = v;
            if (t0 + tr < r.hi && n0 + c8 < p.N) v = *reinterpret_cast<const uint4*>(p.dc + (t0 + tr) * p.N + n0 + c8);
            if (t0 + tr < r.hi && k0 + c8 < p.K) w = *reinterpret_cast<const uint4*>(p.a + (t0 + tr) * p.K + k0 + c8);
            const uint32_t vv[4] = {v.x, v.y, v.z, v.w}, ww[4] = {w.x, w.y, w.z, w.w};
            for (int i = 0; i < 8; ++i) {
                s_n[(c8 + i) * kPitch + tr] = (uint16_t)(vv[i / 2] >> (16 * (i & 1)));
                s_k[(c8 + i) * kPitch + tr] = (uint16_t)(ww[i / 2] >> (16 * (i & 1)));
            }
            __syncthreads();
            v8b fn[2], fk[2];
            for (int i = 0; i < 2; ++i) {
                fn[i] = *reinterpret_cast<const v8b*>(s_n + (wm * 32 + i * 16 + l16) * kPitch + kg * 8);
                fk[i] = *reinterpret_cast<const v8b*>(s_k + (wn * 32 + i * 16 + l16) * kPitch + kg * 8);
            }
            for (int i = 0; i < 2; ++i)
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fk[i], fn[j], acc[i][j], 0, 0, 0);
            if (p.dbias && k0 == 0 && tid < kTile)
                for (int i = 0; i < kDepth; ++i) bsum += bf16_to_f32(s_n[tid * kPitch + i]);
            __syncthreads();
        }
    }
    for (int j = 0; j < 2; ++j) {
        const int64_t n = n0 + wm * 32 + j * 16 + l16;
        if (n >= p.N) continue;
        for (int i = 0; i < 2; ++i) {
            const int64_t k = k0 + wn * 32 + i * 16 + kg * 4;
            if (k >= p.K) continue;
            float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
            uint8_t* at = static_cast<uint8_t*>(p.dw) + ((e * p.N + n) * p.K + k) * (p.dw32 ? 4 : 2);
            if (p.accumulate) {
                float old[4];
                load_n<4>(at, p.dw32, true, 4, old);
                for (int q = 0; q < 4; ++q) v[q] += old[q];
            }
            store_n<4>(at, p.dw32, true, 4, v);
        }
    }
    if (p.dbias && k0 == 0 && tid < kTile && n0 + tid < p.N) {
        float* at = p.dbias + e * p.N + n0 + tid;
        *at = p.accumulate ? *at + bsum : bsum;
    }
}

}  // namespace

hipError_t launch_matmul_bf16_weights(const void* dc, const void* a, void* dw, bool dw32, float* dbias,
                                      bool accumulate, const uint32_t* off, const int32_t* ids, int G, int E,
                                      int64_t T, int64_t N, int64_t K, hipStream_t stream) {
    const WeightsArgs p{static_cast<const uint16_t*>(dc), static_cast<const uint16_t*>(a), dw, dbias, off, ids, G, E,
                        T, N, K, dw32, accumulate};
    const dim3 grid((unsigned)(((N + kTile - 1) / kTile) * ((K + kTile - 1) / kTile)), (unsigned)E);
    hipLaunchKernelGGL(weights_kernel, grid, dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace mxg
