// gemm_bf16.hip -- ragged grouped product of BF16 operands with bias, activation and
// residual in its epilogue, the gradient of its rows through the activation before
// them, and the activation's gradient by itself, for gfx950.
//
//   z[t,n] = sum_k a[t,k] b[e,n,k] + bias[e,n],  c = act(z) + residual
//   da[t,k] = act'(z[t,k]) sum_n dc[t,n] b[e,n,k]
//
// One tile list over all groups: a prefix of the groups' M tiles in LDS gives a workgroup its tiles from their
// numbers, in bands of four M tiles with N outer, so that the workgroups of one XCD share weights and rows
// in its L2.  Two kinds of kernel:
//  * The ring (gemm_bf16_tile.h): one workgroup a CU walks tiles and never drains its loads.  256 x 256 for
//    large products: 1.48 PFLOP/s at 8192^3 (745 us), where a large library product reaches 1.54; bound by the
//    matrix cores at the clock that their power allows (1.7 GHz) and by the stages' loads and fragment reads.
//    With SwiGLU, bias and z kept over 65536 rows of 128 uneven experts 0.95 PFLOP/s: partial tiles, and an
//    epilogue of 9 us a tile whose stores come in bursts.
//  * The split: tiles of 64 x 64 and less, the depth dealt to four or eight waves with a ring each and no
//    barrier until their sums are joined, for products of few tiles: there a stage's latency bounds the time,
//    and each wave has 1/4 or 1/8 of the stages.  128 rows by 4096 x 7168 weights 24 us (2.4 TB/s of weights;
//    128 workgroups, each near what a CU's loads reach), 64 x 64 of 7168 9 us.
// Which one runs is a fit to measured times, beside kRowTiles.
#include "gemm_bf16_tile.h"

namespace mxg {

using namespace bf16;

namespace {

// The tiles of a ragged product: BACK reads the weights wide (its depth is their row
// index) and ends in the backward epilogue.
template <class TL, bool BACK>
struct RowsJob {
    struct Coord {
        int e, rows_in, cols_in, m0, n0, stages, depth;
        const uint8_t *a, *b;
    };
    static constexpr bool kSums = false;
    const Bf16Problem& p;
    const uint32_t* s_pre;  // M tiles before each group, then of all
    const uint32_t* s_off;
    const int32_t* s_ids;
    int ntn, mband;
    Items items;
    int64_t lda, ldb;
    int cols, deep, grid;

    __device__ __forceinline__ bool next(int& W, Coord& c) const {
        for (; W < items.all; W += grid) {
            locate(W, c);
            if (c.cols_in > 0) return true;  // the second half of a narrow last tile has no columns
        }
        return false;
    }
    // The tile of item W: its group by a two-step search of the prefix (64 lanes over
    // every 16th entry, then 16).  Tiles run in bands of mband M tiles, N outer in a band.
    __device__ __forceinline__ void locate(int W, Coord& c) const {
        const bool split = W >= items.full;
        const int L = split ? items.full + (W - items.full) / 2 : W;
        const uint32_t x = (uint32_t)L / (uint32_t)ntn;
        const int lane = fresh_lane(), l16 = lane & 15, G = p.G;
        uint64_t m = __ballot(lane * 16 <= G && s_pre[lane * 16 <= G ? lane * 16 : 0] <= x);
        const int base = (__popcll(m) - 1) * 16, idx = base + l16;
        m = __ballot(lane < 16 && idx <= G && s_pre[idx <= G ? idx : 0] <= x);
        const int g = base + __popcll(m) - 1;
        const int first = (int)s_pre[g], mtiles = (int)s_pre[g + 1] - first;
        const uint32_t local = (uint32_t)(L - first * ntn);
        const int mb = mband < mtiles ? mband : mtiles;
        const int band = (int)(local / (uint32_t)(mb * ntn));
        const uint32_t r = local - (uint32_t)(band * mb * ntn);
        const int left = mtiles - band * mb, gm = left < mb ? left : mb;
        const int nt = (int)(r / (uint32_t)gm), mt = band * mb + (int)r - nt * gm;
        const int64_t lo = (int64_t)s_off[g] < p.T ? (int64_t)s_off[g] : p.T;
        const int64_t hi = (int64_t)s_off[g + 1] < p.T ? (int64_t)s_off[g + 1] : p.T;
        c.e = __builtin_amdgcn_readfirstlane(s_ids[g]);
        c.m0 = __builtin_amdgcn_readfirstlane((int)lo + mt * TL::BM);
        const int rows = (int)hi - c.m0;
        c.rows_in = __builtin_amdgcn_readfirstlane(rows < TL::BM ? rows : TL::BM);
        const int width = split ? TL::BN / 2 : TL::BN;  // half a tile along N
        c.n0 = __builtin_amdgcn_readfirstlane(nt * TL::BN + (split && (W - items.full) % 2 ? TL::BN / 2 : 0));
        c.cols_in = cols - c.n0 < width ? cols - c.n0 : width;
        c.depth = deep;
        c.stages = (deep + kStageDepth - 1) / kStageDepth;
        c.a = static_cast<const uint8_t*>(p.a) + c.m0 * lda;
        c.b = static_cast<const uint8_t*>(p.b) + (int64_t)c.e * p.N * p.K * 2 + c.n0 * (BACK ? 2 : ldb);
    }
    __device__ __forceinline__ bool segment(Coord&) const { return false; }

    template <class>
    __device__ __forceinline__ void finish(const Coord& c, const v4f (&acc)[TL::TN][TL::TM], int wm, int wn,
                                           uint8_t* out) const {
        with_act(p.act, [&](auto act) {
            if constexpr (BACK) {
                put_rows<TL, Before<8>>(
                    acc, wm, wn, c.rows_in, c.cols_in, out,
                    [&](int row, int col, Before<8>& x) { fetch_backward<act(), 8>(p, c.m0 + row, c.n0 + col, x); },
                    [&](int row, int col, const float* v, const Before<8>& x) {
                        finish_backward<act(), 8>(p, c.m0 + row, c.n0 + col, v, x);
                    });
            } else if ((p.N & 7) == 0) {
                put_rows<TL, Beside>(
                    acc, wm, wn, c.rows_in, c.cols_in, out,
                    [&](int row, int col, Beside& x) { fetch8<act(), true>(p, c.e, c.m0 + row, c.n0 + col, x); },
                    [&](int row, int col, const float* v, const Beside& x) {
                        finish8<act(), true>(p, c.m0 + row, c.n0 + col, v, x);
                    });
            } else {
                put_blocks<TL>(acc, wm, wn, c.rows_in, c.cols_in, out, [&](int row, int col, const float* v) {
                    Beside x;
                    fetch8<act(), false>(p, c.e, c.m0 + row, c.n0 + col, x);
                    finish8<act(), false>(p, c.m0 + row, c.n0 + col, v, x);
                });
            }
        });
    }
};

// Indexes of tiles and of their halves are 32 bits wide.
constexpr int kMostTiles = INT32_MAX / 2;

// The routing and the M tiles before each group into LDS; returns how many tiles there are, N tiles and
// all.  Rows with one owner stay below kMostTiles (the launch sees to it).  Offsets that go back need not:
// counted in 64 bits and cut off there, the prefix never falls and each tile has its rows.
template <class TL>
__device__ __forceinline__ int load_groups(const Bf16Problem& p, int ntn, uint32_t* s_pre, uint32_t* s_off,
                                           int32_t* s_ids, uint64_t* s_wave) {
    const int tid = threadIdx.x, G = p.G;
    if (p.off == nullptr) {  // one group
        const int total = (int)((p.T + TL::BM - 1) / TL::BM);
        if (tid == 0) {
            s_off[0] = s_pre[0] = 0;
            s_off[1] = (uint32_t)p.T;
            s_pre[1] = (uint32_t)total;
            s_ids[0] = 0;
        }
        __syncthreads();
        return total * ntn;
    }
    for (int i = tid; i <= G; i += TL::kThreads) {
        s_off[i] = p.off[i];
        if (i < G) s_ids[i] = p.ids[i];
    }
    __syncthreads();
    constexpr int kPer = (kMaxGroups + TL::kThreads - 1) / TL::kThreads;
    const uint64_t most = (uint64_t)(kMostTiles / ntn);
    uint32_t cnt[kPer];
    uint64_t local = 0, total;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int g = tid * kPer + i;
        cnt[i] = 0;
        if (g < G) {
            const GroupRange r = group_range(s_off, s_ids, g, p.T, p.E);
            cnt[i] = (uint32_t)((r.hi - r.lo + TL::BM - 1) / TL::BM);
        }
        local += cnt[i];
    }
    uint64_t before = gemm::block_exclusive_scan<TL::kThreads, uint64_t>(local, s_wave, &total);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int g = tid * kPer + i;
        if (g < G) s_pre[g] = (uint32_t)(before < most ? before : most);
        before += cnt[i];
    }
    total = total < most ? total : most;
    if (tid == 0) s_pre[G] = (uint32_t)total;
    __syncthreads();
    return __builtin_amdgcn_readfirstlane((int)total * ntn);  // in a scalar register (8192^3: 760 us without, 749)
}

template <class TL, bool BACK>
__global__ __launch_bounds__(TL::kThreads, 1) void matmul_bf16_kernel(const Bf16Problem p, int ntn, int mband) {
    __shared__ __attribute__((aligned(512))) uint8_t s_ring[TL::kLds];
    __shared__ uint32_t s_pre[kMaxGroups + 1], s_off[kMaxGroups + 1];
    __shared__ uint64_t s_wave[TL::kWaves];
    __shared__ int32_t s_ids[kMaxGroups];
    const int total = load_groups<TL>(p, ntn, s_pre, s_off, s_ids, s_wave);
    const int cols = (int)(BACK ? p.K : p.N), deep = (int)(BACK ? p.N : p.K), grid = (int)gridDim.x;
    RowsJob<TL, BACK> job{p, s_pre, s_off, s_ids, ntn, mband, items_of(total, grid),
                          (int64_t)deep * 2, (int64_t)(BACK ? cols : deep) * 2, cols, deep, grid};
    run_tiles<TL>(job, s_ring, gemm::xcd_remap((int)blockIdx.x, grid), grid);
}

// Small tiles, their depth split over a workgroup's waves.  One a workgroup: the grid has a tile for each
// that rows with one owner make, as far as a launch holds them.  Offsets that go back make more, the loop's later
// rounds.
template <class TL, bool BACK>
__global__ __launch_bounds__(TL::kThreads, 1) void matmul_bf16_split_kernel(const Bf16Problem p, int ntn) {
    __shared__ __attribute__((aligned(512))) uint8_t s_ring[TL::kLds];
    __shared__ uint32_t s_pre[kMaxGroups + 1], s_off[kMaxGroups + 1];
    __shared__ uint64_t s_wave[TL::kWaves];
    __shared__ int32_t s_ids[kMaxGroups];
    const int total = load_groups<TL>(p, ntn, s_pre, s_off, s_ids, s_wave), grid = (int)gridDim.x;
    const int cols = (int)(BACK ? p.K : p.N), deep = (int)(BACK ? p.N : p.K);
    RowsJob<TL, BACK> job{p, s_pre, s_off, s_ids, ntn, 1 << 20, {total, total},
                          (int64_t)deep * 2, (int64_t)(BACK ? cols : deep) * 2, cols, deep, total};
    for (int64_t W = gemm::xcd_remap((int)blockIdx.x, grid); W < total; W += grid) {  // workgroup-uniform
        typename RowsJob<TL, BACK>::Coord c;
        job.locate((int)W, c);
        with_act(p.act, [&](auto act) {
            run_split<TL>(job, c, s_ring, [&](int row, int col, const float* v) {
                if constexpr (BACK) {
                    Before<8> x;
                    fetch_backward<act(), 8>(p, c.m0 + row, c.n0 + col, x);
                    finish_backward<act(), 8>(p, c.m0 + row, c.n0 + col, v, x);
                } else {
                    Beside x;
                    if ((p.N & 7) == 0) {
                        fetch8<act(), true>(p, c.e, c.m0 + row, c.n0 + col, x);
                        finish8<act(), true>(p, c.m0 + row, c.n0 + col, v, x);
                    } else {
                        fetch8<act(), false>(p, c.e, c.m0 + row, c.n0 + col, x);
                        finish8<act(), false>(p, c.m0 + row, c.n0 + col, v, x);
                    }
                }
            });
        });
        __syncthreads();  // the sums are read before the next tile's loads take their place
    }
}

int64_t compute_units() {
    const int cus = gemm::device_cus();
    return cus > 0 ? cus : 256;
}

template <class TL, bool BACK>
hipError_t launch_tile(const Bf16Problem& p, int mband, hipStream_t stream) {
    const int64_t ntn = ((BACK ? p.K : p.N) + TL::BN - 1) / TL::BN;
    const int64_t groups = p.G < p.T ? p.G : p.T, most = (p.T / TL::BM + groups) * ntn;
    if (most > kMostTiles) return hipErrorInvalidValue;  // more than a device's memory holds
    const int64_t room = compute_units(), grid = most < room ? most : room;
    hipLaunchKernelGGL((matmul_bf16_kernel<TL, BACK>), dim3((unsigned)grid), dim3(TL::kThreads), 0, stream, p,
                       (int)ntn, mband);
    return hipGetLastError();
}

template <class TL, bool BACK>
hipError_t launch_split(const Bf16Problem& p, hipStream_t stream) {
    const int64_t ntn = ((BACK ? p.K : p.N) + TL::BN - 1) / TL::BN;
    const int64_t groups = p.G < p.T ? p.G : p.T, most = (p.T / TL::BM + groups) * ntn;
    if (most > kMostTiles) return hipErrorInvalidValue;  // more than a device's memory holds
    hipLaunchKernelGGL((matmul_bf16_split_kernel<TL, BACK>), dim3(workgroups(most, TL::kThreads)), dim3(TL::kThreads),
                       0, stream, p, (int)ntn);
    return hipGetLastError();
}

// Measured (us a call), the ring kernel's 256 x 256 / 256 x 128 / 128 x 128 / 64 x 128 / 32 x 128 and, with
// the depth split, 64 x 64 / 32 x 32 / 16 x 32:
// dense 4096 x 2048 of 2048: 52 / 39 / 54 / 76 / 104 / 104 / 207 / 315;
// 2048 x 2048 of 2048: 47 / 32 / 26 / 35 / 52 / 58 / 109 / 162;
// 1024 x 2048 of 2048: 46 / 29 / 23 / 19 / 27 / 28 / 51 / 82; 256 x 4096 of 4096: 81 / 52 / 38 / 29 / 24 / 28 / 38 / 59;
// 128 x 4096 of 7168: 105 / 69 / 55 / 45 / 37 / 24 / 36 / 48; 16 x 4096 of 7168: 104 / 67 / 49 / 38 / 36 / 20 / 12 / 19;
// 1 x 4096 of 4096: 62 / 41 / 30 / 24 / 22 / 13 / 7.9 / 6.9; 64 x 64 of 7168: 106 / 69 / 46 / 40 / 34 / 19 / 11 / 8.7;
// 5003 rows of 24 uneven groups, 2080 x 1000: 54 / 59 / 51 / 58 / 80 / 86 / 177 / 265; 512 rows of 8, 4096 x 4096:
// 71 / 56 / 47 / 72 / 71 / 75 / 116 / 164; the rows' gradient of 8192 x 7168 of 64: 37 / 39 / 47 / 72 / 123 / 203 / 603 /
// 1241.
// Tiles of 128 rows and less keep four stages and more in flight: with two, 2048 x 2048 of 2048 in 128 x 128 took 43.
constexpr Candidate kRowTiles[] = {
    {256, 256, 1, 1, 5.0, 1.2, 12.0}, {256, 128, 1, 1, 5.0, 0.59, 12.5}, {128, 128, 1, 1, 4.5, 0.45, 14.0},
    {64, 128, 1, 1, 4.5, 0.35, 14.5}, {32, 128, 1, 1, 3.5, 0.28, 16.0},  {64, 64, 4, 1, 3.0, 0.7, 11.0},
    {32, 32, 4, 1, 3.0, 0.33, 7.5},   {16, 32, 8, 1, 4.0, 0.37, 7.5},
};

int row_tile(const Bf16Problem& p, bool back) {
    const int64_t hint = p.max_rows_hint < p.T ? (p.max_rows_hint > 0 ? p.max_rows_hint : 1) : p.T;
    int64_t groups = p.G < p.T ? p.G : p.T;
    if (groups > 1 + p.T - hint) groups = 1 + p.T - hint;  // the rows beside the largest group's
    return fastest(kRowTiles, {groups, p.T, back ? p.K : p.N, back ? p.N : p.K}, compute_units());
}

template <bool BACK>
hipError_t launch(const Bf16Problem& p, hipStream_t stream) {
    switch (row_tile(p, BACK)) {
        case 0: return launch_tile<Tile<256, 256, 4, 2, 2, false, BACK>, BACK>(p, 4, stream);
        case 1: return launch_tile<Tile<256, 128, 4, 2, 2, false, BACK>, BACK>(p, 4, stream);
        case 2: return launch_tile<Tile<128, 128, 2, 4, 4, false, BACK>, BACK>(p, 4, stream);
        case 3: return launch_tile<Tile<64, 128, 2, 4, 5, false, BACK>, BACK>(p, 1 << 20, stream);
        case 4: return launch_tile<Tile<32, 128, 1, 4, 6, false, BACK>, BACK>(p, 1 << 20, stream);
        case 5: return launch_split<SplitTile<64, 64, 4, 2, false, BACK>, BACK>(p, stream);
        case 6: return launch_split<SplitTile<32, 32, 4, 4, false, BACK>, BACK>(p, stream);
        default: return launch_split<SplitTile<16, 32, 8, 3, false, BACK>, BACK>(p, stream);
    }
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
            swiglu_grad<4>(zv, d, out);
        } else {
            load_n<8>(static_cast<const uint16_t*>(dc) + u * 8, false, true, 8, out);
#pragma unroll
            for (int i = 0; i < 8; ++i) out[i] *= derivative<ACT>(zv[i]);
        }
        store_n<8>(static_cast<uint16_t*>(dz) + u * 8, false, true, 8, out);
    }
}

}  // namespace

int bf16_tile_choice(const Bf16Problem& p, bool back) {
    const Candidate& c = kRowTiles[row_tile(p, back)];
    return 1000 * c.rows + c.cols;
}
hipError_t launch_matmul_bf16(const Bf16Problem& p, hipStream_t stream) { return launch<false>(p, stream); }
hipError_t launch_matmul_bf16_backward(const Bf16Problem& p, hipStream_t stream) { return launch<true>(p, stream); }

hipError_t launch_activation_backward(int act, const void* dc, const void* z, void* dz, int64_t T, int64_t N,
                                      hipStream_t stream) {
    const int64_t units = T * N / (act == kSwiglu ? 4 : 8);
    const dim3 grid(workgroups((units + 255) / 256, 256));
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
