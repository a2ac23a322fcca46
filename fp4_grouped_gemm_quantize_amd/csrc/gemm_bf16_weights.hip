// gemm_bf16_weights.hip -- the gradient of the experts' weights and biases: for each
// expert the product of its rows' gradients, transposed, with its rows, for gfx950.
//
// dw[e,n,k] = sum over expert e's rows t of dc[t,n] a[t,k]: both operands are wide (the
// depth is their row index), so both go through the transposing LDS loads.  A tile's depth
// is its expert's rows, group by group; the tiles of all experts are one list, so that short
// and long ones share the chip, and a tile without rows costs its zeros alone.
//
// Bound by what it writes where experts have few rows (dw in fp32 is 4 N K bytes an expert: 32768 rows of 64
// experts, 1536 x 4096, 685 us, 1.6 GB of dw at 2.4 TB/s beside 0.6 PFLOP/s: an expert's 512 rows are eight
// stages, behind which its tile's stores wait for memory), by the transposing reads and the power where they
// have many (8192^3 840 us, 1.31 PFLOP/s, a library product of the same layout 946).  A router's
// weights (64 x 7168 over 8192 rows) are few tiles with a long depth: split over a workgroup's waves 31 us where the
// caches hold the rows, 48 where each call has others.
// Experts' rows stay in one workgroup, so a repeated call gives the same bits; no atomics, no workspace.
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

template <class TL, bool BIAS>
struct WeightsJob {
    static constexpr bool kSums = BIAS;
    struct Coord {
        int e, g, rows_in, cols_in, n0, k0, stages, depth;  // g: the group of the present segment
        const uint8_t *a, *b;
    };
    const WeightsArgs& p;
    const uint32_t* s_off;   // clamped to T
    const int32_t* s_ids;
    const int32_t* s_order;  // experts, those of most stages first; nullptr: as they are numbered
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
        int L = split ? items.full + (W - items.full) / 2 : W;
        // every other whole round runs backwards, so that what falls along the list is even over the workgroups
        const int round = (int)((uint32_t)L / (uint32_t)grid);
        if ((round & 1) && (round + 1) * grid <= items.full) L = (2 * round + 1) * grid - 1 - L;
        const int tiles = p.ntn * p.ntk, turn = (int)((uint32_t)L / (uint32_t)tiles), local = L - turn * tiles;
        const int e = s_order ? s_order[turn] : turn;
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
        int64_t stages = 0;  // rows that many groups take may come to more than 32 bits
        for (int g = first; g >= 0; g = find(c.e, g + 1)) stages += ((uint32_t)rows(g) + kStageDepth - 1) / kStageDepth;
        c.stages = __builtin_amdgcn_readfirstlane((int)(stages < INT32_MAX / 2 ? stages : INT32_MAX / 2));
        if (first >= 0) begin(c, first);
    }
    __device__ __forceinline__ bool next(int& W, Coord& c) const {
        for (; W < items.all; W += grid) {
            locate(W, c);
            if (c.cols_in > 0) return true;
        }
        return false;
    }
    // dbias: the sums of dc's columns, by one tile of a row of tiles, another in each row (they take
    // longer: the same workgroups would get all of a band's first ones)
    __device__ __forceinline__ bool sums(const Coord& c) const { return c.k0 == c.n0 / TL::BM % p.ntk * TL::BN; }
    __device__ __forceinline__ void put_sum(const Coord& c, int row, float v) const {
        if (p.accumulate && c.stages == 0) return;
        float* at = p.dbias + (int64_t)c.e * p.N + c.n0 + row;
        *at = p.accumulate ? *at + v : v;
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

// Experts by falling number of stages (ties to the lower id).  The tiles of a launch are dealt out in
// rounds, to and fro: in this order the workgroups' shares differ by less than a long tile
// (32768 rows of 64 uneven experts, 1536 x 4096: as numbered 793 us).
__device__ __forceinline__ void order_experts(const WeightsArgs& p, const uint32_t* s_off, const int32_t* s_ids,
                                              uint32_t* s_cost, int32_t* s_order) {
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) s_cost[e] = 0;
    __syncthreads();
    for (int g = threadIdx.x; g < p.G; g += blockDim.x)
        if (s_ids[g] >= 0 && s_ids[g] < p.E && s_off[g] < s_off[g + 1])
            atomicAdd(&s_cost[s_ids[g]], (s_off[g + 1] - s_off[g] + kStageDepth - 1) / kStageDepth);
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        const uint32_t mine = s_cost[e];
        int rank = 0;
        for (int o = 0; o < p.E; ++o) rank += s_cost[o] > mine || (s_cost[o] == mine && o < e);
        s_order[rank] = e;
    }
    __syncthreads();
}

template <class TL, bool BIAS>
__global__ __launch_bounds__(TL::kThreads, 1) void weights_kernel(const WeightsArgs p) {
    __shared__ __attribute__((aligned(512))) uint8_t s_ring[TL::kLds];
    __shared__ uint32_t s_off[kMaxGroups + 1];
    __shared__ int32_t s_ids[kMaxGroups], s_order[kMaxGroups];
    load_groups(p, s_off, s_ids);
    const bool sorted = p.E <= kMaxGroups;
    static_assert(TL::kLds >= 4 * kMaxGroups, "the costs fit the ring");
    if (sorted) order_experts(p, s_off, s_ids, reinterpret_cast<uint32_t*>(s_ring), s_order);
    const int grid = (int)gridDim.x;
    WeightsJob<TL, BIAS> job{p, s_off, s_ids, sorted ? s_order : nullptr, p.N * 2, p.K * 2,
                             items_of(p.E * p.ntn * p.ntk, grid), grid, 4};
    run_tiles<TL>(job, s_ring, gemm::xcd_remap((int)blockIdx.x, grid), grid);
}

// Small tiles, one a workgroup, their depth split over its waves.
template <class TL, bool BIAS>
__global__ __launch_bounds__(TL::kThreads, 1) void weights_split_kernel(const WeightsArgs p) {
    __shared__ __attribute__((aligned(512))) uint8_t s_ring[TL::kLds];
    __shared__ uint32_t s_off[kMaxGroups + 1];
    __shared__ int32_t s_ids[kMaxGroups];
    load_groups(p, s_off, s_ids);
    const int items = p.E * p.ntn * p.ntk;
    WeightsJob<TL, BIAS> job{p, s_off, s_ids, nullptr, p.N * 2, p.K * 2, {items, items}, items, 4};
    const int grid = (int)gridDim.x;
    for (int64_t W = gemm::xcd_remap((int)blockIdx.x, grid); W < items; W += grid) {  // workgroup-uniform
        typename WeightsJob<TL, BIAS>::Coord c;
        job.locate((int)W, c);
        if (p.accumulate && c.stages == 0) continue;
        run_split<TL>(job, c, s_ring, [&](int row, int col, const float* v) {
            Old<8> old;
            fetch(p, c.e, c.n0 + row, c.k0 + col, old);
            write(p, c.e, c.n0 + row, c.k0 + col, v, old);
        });
        __syncthreads();  // the sums are read before the next tile's loads take their place
    }
}

int64_t compute_units() {
    const int cus = gemm::device_cus();
    return cus > 0 ? cus : 256;
}

// Measured (us a call; 256 and 128 rows in the ring kernel, 64 x 64 and 64 x 32 with the depth split):
// 32768 rows of 64 uneven experts, 1536 x 4096: 684 / 1147 / 2629 / 4606; 8192 rows, 4096 x 7168: 443 / 698 / 767 /
// 1333; 16384 rows of 8, 256 x 2048: 61 / 37 / 41 / 67; 4096 rows, 512 x 1024: 103 / 60 / 18 / 16; 8192 rows,
// 64 x 7168: 164 / 110 / 33 / 31 (one call by itself behind a write of 1 GiB, its launch with it: 76 and 67 for the last
// two); 5003 rows of 24, 1000 x 2080: 93 / 128 / 290 / 482.
constexpr Candidate kWeightTiles[] = {
    {256, 256, 1, 1, 12.0, 1.1, 12.0}, {128, 128, 1, 2, 6.0, 0.6, 11.0}, {64, 64, 4, 1, 3.0, 0.95, 11.0},
    {64, 32, 4, 1, 3.0, 0.87, 12.6},
};

int weight_tile(int G, int E, int64_t T, int64_t N, int64_t K) {
    // The experts that may have rows, as one output: N rows each, filled up to whole tiles, and a depth
    // of their share of the rows.
    int64_t used = G < T ? G : T;
    used = used < E ? (used > 0 ? used : 1) : E;
    int best = 0;
    double least = 0.0;
    const int n = sizeof kWeightTiles / sizeof kWeightTiles[0];
    for (int i = 0; i < n; ++i) {
        const Candidate& c = kWeightTiles[i];
        const int64_t rows = (N + c.rows - 1) / c.rows * c.rows * used;
        const double t = time_of(c, {1, rows, K, T / used}, compute_units());
        if (i == 0 || t < least) {
            best = i;
            least = t;
        }
    }
    return best;
}

}  // namespace

int bf16_weights_tile_choice(int G, int E, int64_t T, int64_t N, int64_t K) {
    const Candidate& c = kWeightTiles[weight_tile(G, E, T, N, K)];
    return 1000 * c.rows + c.cols;
}

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
    auto split = [&](auto tile, auto bias) {
        using TL = decltype(tile);
        const int64_t n = tiles(TL::BM, TL::BN);
        if (n > INT32_MAX) return hipErrorInvalidValue;  // more than a device's memory holds
        hipLaunchKernelGGL((weights_split_kernel<TL, decltype(bias)::value>), dim3(workgroups(n, TL::kThreads)),
                           dim3(TL::kThreads), 0, stream, p);
        return hipGetLastError();
    };
    auto whole = [&](auto tile, auto bias, int per_cu) {
        using TL = decltype(tile);
        const int64_t n = tiles(TL::BM, TL::BN), room = compute_units() * per_cu;
        if (2 * n > INT32_MAX) return hipErrorInvalidValue;
        hipLaunchKernelGGL((weights_kernel<TL, decltype(bias)::value>), dim3((unsigned)(n < room ? n : room)),
                           dim3(TL::kThreads), 0, stream, p);
        return hipGetLastError();
    };
    auto pick = [&](auto bias) {
        switch (weight_tile(G, E, T, N, K)) {
            case 0: return whole(Tile<256, 256, 4, 2, 2, true, true>{}, bias, 1);
            case 1: return whole(Tile<128, 128, 2, 2, 2, true, true>{}, bias, 2);
            case 2: return split(SplitTile<64, 64, 4, 2, true, true>{}, bias);
            default: return split(SplitTile<64, 32, 4, 3, true, true>{}, bias);
        }
    };
    return dbias ? pick(std::true_type{}) : pick(std::false_type{});
}

}  // namespace mxg
