// gemm_bf16_weights.hip -- the gradient of the experts' weights and biases: for each
// expert the product of its rows' gradients, transposed, with its rows, for gfx950.
//
// dw[e,n,k] = sum over expert e's rows t of dc[t,n] a[t,k]: both operands are wide (the
// depth is their row index), so both go through the transposing LDS loads.  A tile's depth
// is its expert's rows, group by group; the tiles of all experts are one list, so that short
// and long ones share the chip, and a tile without rows costs its zeros alone.
#include <stdlib.h>

#include "gemm_bf16_tile.h"

namespace mxg {

using namespace bf16;

namespace {

struct WeightsArgs {
    const uint8_t* dc;
    const uint8_t* a;
    void* dw;
    float* dbias;
    const uint32_t* off;
    const int32_t* ids;
    int G, E;
    int64_t T, N, K;
    bool dw32, accumulate;
    int ntn, ntk;  // tiles along N and K
};

// W neighbouring columns of dw out; old: what they held, asked for ahead.
template <int W>
struct Old {
    float v[W];
};
__device__ __forceinline__ uint8_t* dw_at(const WeightsArgs& p, int e, int64_t n, int64_t k) {
    return static_cast<uint8_t*>(p.dw) + (((int64_t)e * p.N + n) * p.K + k) * (p.dw32 ? 4 : 2);
}
template <int W>
__device__ __forceinline__ void fetch(const WeightsArgs& p, int e, int64_t n, int64_t k, Old<W>& old) {
    if (p.accumulate) load_n<W>(dw_at(p, e, n, k), p.dw32, true, W, old.v);
}
template <int W>
__device__ __forceinline__ void write(const WeightsArgs& p, int e, int64_t n, int64_t k, const float* sums,
                                       const Old<W>& old) {
    float v[W];
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = p.accumulate ? sums[i] + old.v[i] : sums[i];
    store_n<W>(dw_at(p, e, n, k), p.dw32, true, W, v);
}

template <class TL>
struct WeightsJob {
    struct Coord {
        int e, g, rows_in, cols_in, n0, k0, stages, depth;  // g: the group of the present segment
        const uint8_t *a, *b;
    };
    const WeightsArgs& p;
    const uint32_t* s_off;  // clamped to T
    const int32_t* s_ids;
    int64_t lda, ldb;
    Items items;
    int grid, mband;

    // The first group of expert e from g on that has rows, or -1.
    __device__ __forceinline__ int find(int e, int g) const {
        int found = -1;
        for (; found < 0 && g < p.G; g += kWave) {
            const int i = g + (int)(threadIdx.x & (kWave - 1)), j = i < p.G ? i : 0;
            const uint64_t m = __ballot(i < p.G && s_ids[j] == e && s_off[j] < s_off[j + 1]);
            found = __builtin_amdgcn_readfirstlane(m ? g + __builtin_ctzll(m) : -1);
        }
        return found;
    }
    __device__ __forceinline__ int rows(int g) const {
        return __builtin_amdgcn_readfirstlane((int)(s_off[g + 1] - s_off[g]));
    }
    __device__ __forceinline__ void begin(Coord& c, int g) const {
        c.g = g;
        c.depth = rows(g);
        const int64_t lo = (int64_t)(uint32_t)__builtin_amdgcn_readfirstlane(s_off[g]);
        c.a = p.dc + lo * lda + c.n0 * 2;
        c.b = p.a + lo * ldb + c.k0 * 2;
    }
    __device__ __forceinline__ bool segment(Coord& c) const {
        const int g = find(c.e, c.g + 1);
        if (g < 0) return false;
        begin(c, g);
        return true;
    }

    __device__ __forceinline__ void locate(int W, Coord& c) const {
        const bool split = W >= items.full;
        const int L = split ? items.full + (W - items.full) / 2 : W, tiles = p.ntn * p.ntk;
        const int e = (int)((uint32_t)L / (uint32_t)tiles), local = L - e * tiles;
        const int mb = mband < p.ntn ? mband : p.ntn;  // bands of mband tiles along N, K walked within one
        const int band = (int)((uint32_t)local / (uint32_t)(mb * p.ntk)), r = local - band * mb * p.ntk;
        const int left = p.ntn - band * mb, gm = left < mb ? left : mb, kt = (int)((uint32_t)r / (uint32_t)gm);
        c.e = __builtin_amdgcn_readfirstlane(e);
        c.n0 = __builtin_amdgcn_readfirstlane((band * mb + r - kt * gm) * TL::BM);
        c.k0 = __builtin_amdgcn_readfirstlane(kt * TL::BN + (split && (W - items.full) % 2 ? TL::BN / 2 : 0));
        const int width = split ? TL::BN / 2 : TL::BN, rows_left = (int)p.N - c.n0, cols_left = (int)p.K - c.k0;
        c.rows_in = rows_left < TL::BM ? rows_left : TL::BM;
        c.cols_in = cols_left < width ? cols_left : width;
        const int first = find(c.e, 0);
        int stages = 0;
        for (int g = first; g >= 0; g = find(c.e, g + 1)) stages += (rows(g) + kStageDepth - 1) / kStageDepth;
        c.stages = __builtin_amdgcn_readfirstlane(stages);
        if (first >= 0) begin(c, first);
    }
    __device__ __forceinline__ bool next(int& W, Coord& c) const {
        for (; W < items.all; W += grid) {
            locate(W, c);
            if (c.cols_in > 0) return true;
        }
        return false;
    }
    template <class>
    __device__ __forceinline__ void finish(const Coord& c, const v4f (&acc)[TL::TN][TL::TM], int wm, int wn,
                                           uint8_t* out) const {
        if (p.accumulate && c.stages == 0) return;
        put_rows<TL, Old<8>>(
            acc, wm, wn, c.rows_in, c.cols_in, out,
            [&](int row, int col, Old<8>& old) { fetch(p, c.e, c.n0 + row, c.k0 + col, old); },
            [&](int row, int col, const float* v, const Old<8>& old) {
                write(p, c.e, c.n0 + row, c.k0 + col, v, old);
            });
    }
};

__device__ __forceinline__ void load_groups(const WeightsArgs& p, uint32_t* s_off, int32_t* s_ids) {
    for (int i = threadIdx.x; i <= p.G; i += blockDim.x) {
        const uint32_t o = p.off ? p.off[i] : i ? (uint32_t)p.T : 0;
        s_off[i] = (int64_t)o < p.T ? o : (uint32_t)p.T;
        if (i < p.G) s_ids[i] = p.ids ? p.ids[i] : 0;
    }
    __syncthreads();
}

template <class TL>
__global__ __launch_bounds__(TL::kThreads, 1) void weights_kernel(const WeightsArgs p) {
    __shared__ __attribute__((aligned(512))) uint8_t s_ring[TL::kLds];
    __shared__ uint32_t s_off[kMaxGroups + 1];
    __shared__ int32_t s_ids[kMaxGroups];
    load_groups(p, s_off, s_ids);
    const int grid = (int)gridDim.x;
    WeightsJob<TL> job{p, s_off, s_ids, p.N * 2, p.K * 2, items_of(p.E * p.ntn * p.ntk, grid), grid, 4};
    run_tiles<TL>(job, s_ring, gemm::xcd_remap((int)blockIdx.x, grid), grid);
}

// Small tiles, one a workgroup, their depth split over its waves.
template <class TL>
__global__ __launch_bounds__(TL::kThreads, 1) void weights_split_kernel(const WeightsArgs p) {
    __shared__ __attribute__((aligned(512))) uint8_t s_ring[TL::kLds];
    __shared__ uint32_t s_off[kMaxGroups + 1];
    __shared__ int32_t s_ids[kMaxGroups];
    load_groups(p, s_off, s_ids);
    const int items = p.E * p.ntn * p.ntk;
    WeightsJob<TL> job{p, s_off, s_ids, p.N * 2, p.K * 2, {items, items}, 1, 4};
    typename WeightsJob<TL>::Coord c;
    job.locate(gemm::xcd_remap((int)blockIdx.x, (int)gridDim.x), c);
    if (p.accumulate && c.stages == 0) return;
    run_split<TL>(job, c, s_ring, [&](int row, int col, const float* v) {
        Old<8> old;
        fetch(p, c.e, c.n0 + row, c.k0 + col, old);
        write(p, c.e, c.n0 + row, c.k0 + col, v, old);
    });
}

// dbias: 64 columns of one expert a workgroup, its rows over 16 waves of 8 rows each.
constexpr int kBiasWaves = 16;
__global__ __launch_bounds__(kBiasWaves * kWave) void bias_kernel(const WeightsArgs p) {
    __shared__ float s[kBiasWaves][8][64];
    const int e = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int64_t n = (int64_t)blockIdx.x * 64 + (lane % 8) * 8;
    float sum[8] = {};
    bool any = false;
    for (int g = 0; g < p.G; ++g) {
        if (expert_of(p.ids, g) != e) continue;
        const GroupRange r = rows_of(p.off, p.ids, g, p.T, p.E);
        any = any || r.lo < r.hi;
#pragma unroll 4
        for (int64_t t = r.lo + wave * 8 + lane / 8; t < r.hi; t += kBiasWaves * 8)
            if (n < p.N) {
                float v[8];
                unpack8(*reinterpret_cast<const uint4*>(p.dc + (t * p.N + n) * 2), v);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] += v[i];
            }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s[wave][lane / 8][(lane % 8) * 8 + i] = sum[i];
    __syncthreads();
    if (wave == 0) {
        float v = 0.0f;
        for (int w = 0; w < kBiasWaves; ++w)
#pragma unroll
            for (int i = 0; i < 8; ++i) v += s[w][i][lane];
        const int64_t at = (int64_t)blockIdx.x * 64 + lane;
        if (at < p.N) {
            float* d = p.dbias + (int64_t)e * p.N + at;
            *d = p.accumulate ? *d + v : v;
        }
    }
}

int64_t compute_units() {
    const int cus = gemm::device_cus();
    return cus > 0 ? cus : 256;
}

}  // namespace

hipError_t launch_matmul_bf16_weights(const void* dc, const void* a, void* dw, bool dw32, float* dbias,
                                      bool accumulate, const uint32_t* off, const int32_t* ids, int G, int E,
                                      int64_t T, int64_t N, int64_t K, hipStream_t stream) {
    WeightsArgs p{static_cast<const uint8_t*>(dc), static_cast<const uint8_t*>(a), dw, dbias, off, ids, G, E,
                  T, N, K, dw32, accumulate, 0, 0};
    auto tiles = [&](int BM, int BN) {
        p.ntn = (int)((N + BM - 1) / BM);
        p.ntk = (int)((K + BN - 1) / BN);
        return (int64_t)E * p.ntn * p.ntk;
    };
    const char* f = getenv("MXG_BF16_WTILE");
    const int t = f ? atoi(f) : 256;
    if (t == 64) {
        using TL = SplitTile<64, 64, 4, true, true>;
        const int64_t n = tiles(64, 64);
        hipLaunchKernelGGL(weights_split_kernel<TL>, dim3((unsigned)n), dim3(TL::kThreads), 0, stream, p);
    } else if (t == 32) {
        using TL = SplitTile<64, 32, 5, true, true>;
        const int64_t n = tiles(64, 32);
        hipLaunchKernelGGL(weights_split_kernel<TL>, dim3((unsigned)n), dim3(TL::kThreads), 0, stream, p);
    } else if (t == 128) {
        using TL = Tile<128, 128, 2, 2, true, true>;
        const int64_t n = tiles(128, 128), room = compute_units() * 2;
        hipLaunchKernelGGL(weights_kernel<TL>, dim3((unsigned)(n < room ? n : room)), dim3(TL::kThreads), 0, stream, p);
    } else {
        using TL = Tile<256, 256, 4, 2, true, true>;
        const int64_t n = tiles(256, 256), room = compute_units();
        hipLaunchKernelGGL(weights_kernel<TL>, dim3((unsigned)(n < room ? n : room)), dim3(TL::kThreads), 0, stream, p);
    }
    if (dbias)
        hipLaunchKernelGGL(bias_kernel, dim3((unsigned)((N + 63) / 64), (unsigned)E), dim3(kBiasWaves * kWave), 0,
                           stream, p);
    return hipGetLastError();
}

}  // namespace mxg
