// gemm_block128.hip -- ragged grouped GEMM of FP8 e4m3 operands with an fp32
// scale per 1 x 128 block of A and 128 x 128 block of the weights, BF16 out, for
// gfx950.
//
// (grouped_matmul_rowwise_dynamic_scaled_fp8 with block scales:
//  out[t,n] = sum_b a_scale[t,b] b_scale[e,n/128,b] sum_{k in b} a[t,k] b[e,n,k].)
//
// Design (CDNA4):
//  * Matrix core: v_mfma_f32_16x16x128_f8f6f4, whose depth is one scale block:
//    each block's product leaves the matrix core once, from a zero
//    accumulator, and is added under its scale by one fp32 FMA per element.
//    (The scaled form takes only powers of two.)  The FMAs are half the matrix
//    cores' issue time and run beside them, three products behind.
//  * Operands trade places: the weights are the instruction's A, the tokens its
//    B, so a lane's four results are four columns of one token.  A lane then
//    needs one scale per 16-token block (the token's times the wave's weight
//    scale, which is uniform), and its results pack to 8 bytes of BF16.
//  * K streams in stages of 128 bytes per row (one scale block) through a ring
//    of LDS slots filled by direct global->LDS loads (lds_dma16: the compiler
//    sees no LDS write and adds no waits), the scales beside them, eight blocks
//    of every row at a time.  The ring runs across tiles: while the last stages
//    of a tile are computed the first ones of the next are already on their
//    way, and the epilogue uses only the slot just consumed.
//  * Ragged groups without host sync, XCD-aware order and the persistent
//    schedule as in the rowwise GEMM (gemm_common.h); offsets, ids and the tile
//    prefix are kept in LDS, so finding the next tile costs two LDS reads.
#include <type_traits>

#include "gemm_common.h"

namespace mxg {

using namespace gemm;

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
constexpr int kSB = 128;          // stage bytes per row: one scale block

// BM tokens x BN columns, WGM x WGN waves, SLOTS ring slots (loads run SLOTS - 1
// stages ahead; the wait at a stage's end leaves only those issued in that stage in
// flight, so past the third slot they are early rather than more), SCL scale blocks
// per LDS chunk.
template <int BM_, int BN_, int WGM_, int WGN_, int SLOTS_, int SCL_>
struct BTile {
    static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, kSlots = SLOTS_, kScl = SCL_;
    static constexpr int kWaves = WGM * WGN, kThreads = kWave * kWaves;
    static constexpr int WTM = BM / WGM, WTN = BN / WGN;
    static constexpr int TM = WTM / 16, TN = WTN / 16;
    static_assert(128 % WTN == 0, "a wave's columns lie in one weight scale block");
    static_assert(BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0, "loader: whole row groups per wave");
    static_assert(kWaves % 2 == 0, "per-lane chunk independent of the load index");
};

// A direct-to-LDS load of 4 bytes per lane (lane l at lds + 4 l); see lds_dma16.
__device__ __forceinline__ void lds_dma4(const void* base_in, uint32_t voff, uint32_t lds_in) {
    const uint64_t b = (uint64_t)base_in;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)b);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
    const uint64_t base = ((uint64_t)hi << 32) | (uint64_t)lo;
    const uint32_t lds = (uint32_t)__builtin_amdgcn_readfirstlane(lds_in);
    uint32_t saved_m0;
    __asm__ volatile(
        "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 4\n\t"
        "global_load_lds_dword %1, %2\n\ts_mov_b32 m0, %0"
        : "=&s"(saved_m0)
        : "v"(voff), "s"(base), "s"(lds)
        : "memory");
}

// N direct-to-LDS loads of 16 bytes per lane, load j to lds + 1024 NW j (the lanes
// of this wave side by side), in one block: the first s_nop gives a base written
// by a vector instruction its wait states, the others M0 its own.
template <int N, int STRIDE>
__device__ __forceinline__ void lds_dma16_rows(const void* base_in, const uint32_t (&off)[N], uint32_t lds_in) {
    const uint64_t b = (uint64_t)base_in;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)b);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
    const uint64_t base = ((uint64_t)hi << 32) | (uint64_t)lo;
    const uint32_t lds = (uint32_t)__builtin_amdgcn_readfirstlane(lds_in);
    static_assert(N == 1 || N == 2 || N == 4, "loads per block");
    if constexpr (N == 1)
        __asm__ volatile(
            "s_mov_b32 m0, %2\n\ts_nop 4\n\t"
            "global_load_lds_dwordx4 %0, %1"
            :
            : "v"(off[0]), "s"(base), "s"(lds)
            : "memory", "m0");
    else if constexpr (N == 2)
        __asm__ volatile(
            "s_mov_b32 m0, %3\n\ts_nop 4\n\t"
            "global_load_lds_dwordx4 %0, %2\n\ts_add_u32 m0, m0, %4\n\ts_nop 0\n\t"
            "global_load_lds_dwordx4 %1, %2"
            :
            : "v"(off[0]), "v"(off[1]), "s"(base), "s"(lds), "n"(STRIDE)
            : "memory", "m0", "scc");
    else
        __asm__ volatile(
            "s_mov_b32 m0, %5\n\ts_nop 4\n\t"
            "global_load_lds_dwordx4 %0, %4\n\ts_add_u32 m0, m0, %6\n\ts_nop 0\n\t"
            "global_load_lds_dwordx4 %1, %4\n\ts_add_u32 m0, m0, %6\n\ts_nop 0\n\t"
            "global_load_lds_dwordx4 %2, %4\n\ts_add_u32 m0, m0, %6\n\ts_nop 0\n\t"
            "global_load_lds_dwordx4 %3, %4"
            :
            : "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3]), "s"(base), "s"(lds), "n"(STRIDE)
            : "memory", "m0", "scc");
}

// The lane number.  FRESH: made anew where it is needed, so that what derives from
// it (loader rows, fragment addresses) holds no register between stages: for a wave
// of 128 accumulators, 225 registers instead of 256 (65536 uneven rows 516 -> 500 us,
// 8192^3 490 -> 480).  Smaller tiles have registers to spare and keep it (made anew,
// 128-row tiles 122 -> 126 us on 8192 rows of 32 groups, 32-row tiles 22.2 -> 24.4).
template <bool FRESH>
__device__ __forceinline__ int lane_id() {
    if constexpr (!FRESH) return threadIdx.x & (kWave - 1);
    int l;
    __asm__ volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(l));
    return l;
}

__device__ __forceinline__ v4f mma128(const v8i& n, const v8i& t) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(n, t, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

template <class TL>
__global__ __launch_bounds__(TL::kThreads, 1) void block128_kernel(const GemmArgs args) {
    constexpr int BM = TL::BM, BN = TL::BN, NW = TL::kWaves, NT = TL::kThreads;
    constexpr int WTM = TL::WTM, WTN = TL::WTN, TM = TL::TM, TN = TL::TN;
    constexpr int kSlots = TL::kSlots, kAhead = kSlots - 1, kSclBlocks = TL::kScl;
    constexpr int kAStage = BM * kSB, kBStage = BN * kSB, kStage = kAStage + kBStage;
    constexpr int A_J = BM / 8 / NW, B_J = BN / 8 / NW;
    constexpr int kNBlk = BN / 128;                // weight scale blocks across the tile
    constexpr int kSclA = BM * kSclBlocks * 4;     // bytes of a chunk of A's scales, row by row
    constexpr int kScl = kSclA + 256;              // the weights' after them (64 lanes' worth)
    constexpr int S_J = kSclA / 256 / NW;          // 4-byte loads per wave per chunk (and one for the weights')
    static_assert(kSclA % (256 * NW) == 0 && kNBlk * kSclBlocks <= 64, "scale chunk: whole loads per wave");
    __shared__ __attribute__((aligned(16))) uint8_t s_ring[kSlots * kStage];
    __shared__ __attribute__((aligned(16))) uint8_t s_scl[kSlots * kScl];
    // offsets and ids beside the prefix where LDS has room for them
    constexpr bool kTables = kSlots * (kStage + kScl) + 3 * 4 * (kMaxGroups + 1) + 64 <= 160 * 1024;
    __shared__ uint32_t s_pre[kMaxGroups + 1], s_off[kTables ? kMaxGroups + 1 : 1];
    __shared__ int32_t s_ids[kTables ? kMaxGroups : 1];
    __shared__ uint32_t s_wave[NW];

    constexpr bool kFresh = TM * TN * 4 >= 128;
    // Rows a multiple of 4096 bytes apart begin in the same memory channels, and tiles
    // side by side walk them in step: there each expert begins at a block of its own
    // (such K have no short last block).  For the 128-row tile, which the sizes bound
    // by the weights get: 4096 rows of 64 experts, 4096 x 2048, 137 -> 108 us; the
    // 256-row tile gains nothing (65536 rows) or loses 2 % (8192^3).  The sum of a
    // row's blocks is then in an order that goes by the expert's id.
    constexpr bool kTurn = BM == 128;
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / TL::WGN, wn = wave % TL::WGN;
    const int G = args.G;

    if constexpr (kTables)
        for (int i = tid; i <= G; i += NT) {
            s_off[i] = args.off[i];
            if (i < G) s_ids[i] = args.ids[i];
        }
    const uint32_t* off = kTables ? s_off : args.off;
    const int32_t* ids = kTables ? s_ids : args.ids;
    build_tile_prefix<NT, BM>(args, s_pre, s_wave);  // ends with a barrier
    const int64_t K = args.K;
    const int nkt = (int)((K + kSB - 1) / kSB);
    const int nnb = (int)((args.N + 127) / 128);
    const WorkSplit ws = work_split((int64_t)s_pre[G] * args.ntiles_n, gridDim.x);

    // ---- the tile of work item W: its group by a two-step search of the prefix
    // (64 lanes over every 16th entry, then 16), all from LDS
    struct Coord {
        int e, rows_in, cols_in;
        int64_t m0, n0;
    };
    auto locate = [&](int64_t W) {
        const bool split = W >= ws.full;
        const int64_t L = split ? ws.full + (W - ws.full) / 2 : W;
        const int64_t ntn = args.ntiles_n;
        const uint32_t x = (uint32_t)(L / ntn);  // M tile of the launch
        const int lane = lane_id<kFresh>(), l16 = lane & 15;
        uint64_t m = __ballot(lane * 16 <= G && s_pre[lane * 16 <= G ? lane * 16 : 0] <= x);
        const int base = (__popcll(m) - 1) * 16;
        const int idx = base + l16;
        m = __ballot(lane < 16 && idx <= G && s_pre[idx <= G ? idx : 0] <= x);
        const int g = base + __popcll(m) - 1;
        const int first = (int)s_pre[g], mtiles = (int)s_pre[g + 1] - first;
        const int64_t local = L - first * ntn;
        const int mb = args.mband < mtiles ? args.mband : mtiles;  // tiles run in bands of mb M tiles, N outer
        const int band = (int)(local / (mb * ntn));
        const int64_t r = local - band * mb * ntn;
        const int left = mtiles - band * mb, gm = left < mb ? left : mb;
        const int64_t lo = (int64_t)off[g] < args.T ? (int64_t)off[g] : args.T;
        const int64_t hi = (int64_t)off[g + 1] < args.T ? (int64_t)off[g + 1] : args.T;
        Coord c;
        c.e = __builtin_amdgcn_readfirstlane(ids[g]);
        c.m0 = first_lane64(lo + (int64_t)(band * mb + (int)(r % gm)) * BM);
        c.rows_in = __builtin_amdgcn_readfirstlane((int)(hi - c.m0 < BM ? hi - c.m0 : BM));
        int64_t n0 = r / gm * BN;
        int width = BN;
        if (split) {  // half a tile along N
            width = BN / 2;
            if ((W - ws.full) % 2) n0 += BN / 2;
        }
        c.n0 = first_lane64(n0);
        const int64_t cols = args.N - c.n0;
        c.cols_in = __builtin_amdgcn_readfirstlane((int)(cols < width ? cols : width));
        return c;
    };
    // the next item with columns, from W on (the second half of a narrow last
    // tile has none); W past the end: no more work
    auto next_item = [&](int64_t& W, Coord& c) {
        for (; W < ws.items; W += gridDim.x) {
            c = locate(W);
            if (c.cols_in > 0) return;
        }
    };

    // ---- the producer: stages of tile `pc`, kAhead stages before they are used
    int64_t pw = xcd_remap(blockIdx.x, gridDim.x);
    Coord pc{};
    next_item(pw, pc);
    int pk = 0;          // its next stage
    int pfirst = 0;      // the block of K its stages begin with
    int pslot = 0;       // ring slot that stage goes to
    int pchunk = 0;      // scale buffer of its chunk
    const int ring0 = (int)lds_addr(s_ring), scl0 = (int)lds_addr(s_scl);
    uint32_t a_off[A_J], b_off[B_J];
    const uint8_t *p_a = nullptr, *p_b = nullptr;  // the tile's operands at the producer's stage
    auto set_tile = [&]() {
        const int lane = lane_id<kFresh>();
        const int r0 = wave * 8 + lane / 8;              // row of this lane in load 0 (+ 8 NW per load)
        const int chunk = swz_chunk<kSB>(r0, lane % 8);  // 16-byte piece it fetches: the swizzle
        if constexpr (kTurn) pfirst = K % 4096 == 0 ? pc.e % nkt : 0;
        p_a = args.a + pc.m0 * K + pfirst * kSB;
        p_b = args.b + ((int64_t)pc.e * args.N + pc.n0) * K + pfirst * kSB;
        // rows past the group and columns past N re-read the last real one
#pragma unroll
        for (int j = 0; j < A_J; ++j) {
            const int r = r0 + 8 * NW * j;
            a_off[j] = (uint32_t)(r < pc.rows_in ? r : pc.rows_in - 1) * (uint32_t)K + chunk * 16;
        }
#pragma unroll
        for (int j = 0; j < B_J; ++j) {
            const int r = r0 + 8 * NW * j;
            b_off[j] = (uint32_t)(r < pc.cols_in ? r : pc.cols_in - 1) * (uint32_t)K + chunk * 16;
        }
    };
    // Issue the producer's next stage; returns the number of loads this wave issued.
    auto produce_issue = [&]() -> int {
        if (pw >= ws.items) return 0;
        if (pk == 0) set_tile();
        if (pk == nkt - 1 && K % kSB != 0) {
            // pieces past the end of K fetch the stage's first one instead; the consumer zeroes them
            const int lane = lane_id<kFresh>(), chunk = swz_chunk<kSB>(wave * 8 + lane / 8, lane % 8);
            const uint32_t back = (int64_t)pk * kSB + chunk * 16 < K ? 0 : chunk * 16;
#pragma unroll
            for (int j = 0; j < A_J; ++j) a_off[j] -= back;
#pragma unroll
            for (int j = 0; j < B_J; ++j) b_off[j] -= back;
        }
        // (the A loads end where the B loads begin: kAStage is A_J loads of every wave)
        const int slot = ring0 + pslot * kStage + wave * 1024;
        lds_dma16_rows<A_J, NW * 1024>(p_a, a_off, slot);
        lds_dma16_rows<B_J, NW * 1024>(p_b, b_off, slot + kAStage);
        // around the end of K (where nothing turns this is the tile's end: unused)
        const int64_t step = kTurn && pk + pfirst + 1 == nkt ? kSB - K : kSB;
        p_a += step;
        p_b += step;
        int issued = A_J + B_J;
        if (pk % kSclBlocks == 0) {
            pchunk = pchunk + 1 < kSlots ? pchunk + 1 : 0;
            const int dst = scl0 + pchunk * kScl;
            // kSclBlocks blocks of each of 64 / kSclBlocks rows per load
            const int lane = lane_id<kFresh>(), turn = pk + pfirst + lane % kSclBlocks;
            const int blk = kTurn && turn >= nkt ? turn - nkt : turn;  // past the last without a turn: not used
            const uint32_t col = (uint32_t)(blk < nkt ? blk : nkt - 1);
            const float* as = static_cast<const float*>(args.as) + pc.m0 * nkt;
#pragma unroll
            for (int j = 0; j < S_J; ++j) {
                const int r = (wave + NW * j) * (kWave / kSclBlocks) + lane / kSclBlocks;
                const uint32_t row = (uint32_t)(r < pc.rows_in ? r : pc.rows_in - 1);
                lds_dma4(as, (row * (uint32_t)nkt + col) * 4, dst + (wave + NW * j) * 256);
            }
            // the weights' scales: block row lane / kSclBlocks of the tile (every wave issues the same load)
            const int nb = (int)(pc.n0 / 128) + lane / kSclBlocks;
            const uint32_t brow = (uint32_t)((nb < nnb ? nb : nnb - 1) - (int)(pc.n0 / 128));
            lds_dma4(static_cast<const float*>(args.bs) + ((int64_t)pc.e * nnb + pc.n0 / 128) * nkt,
                     (brow * (uint32_t)nkt + col) * 4, dst + kSclA);
            issued += S_J + 1;
        }
        return issued;
    };
    auto produce_next = [&]() {
        if (pw >= ws.items) return;
        pslot = pslot + 1 < kSlots ? pslot + 1 : 0;
        if (++pk == nkt) {
            pk = 0;
            pw += gridDim.x;
            next_item(pw, pc);
        }
    };
    constexpr int L = A_J + B_J;

    // ---- the consumer
    int64_t cw = pw;
    Coord cc = pc;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        produce_issue();
        produce_next();
    }
    // Waves w and w + 4 share a SIMD.  The upper half issues its loads of a stage
    // behind its first products instead of before its fragment reads, so that one
    // wave of a SIMD multiplies while the other issues loads and waits for its
    // fragments (3 % less time for the 256-row tiles on 65536 uneven rows, 6 % for
    // the 128-row tiles on 5003; behind the 8th product 2 % more, all waves so 6 %
    // more; reading the next stage's fragments behind the last products: no gain).
    constexpr int kLate = 3;
    const bool late = NW == 8 && wave >= NW / 2;
    stage_barrier<0>();
    int cslot = 0, cchunk = 0;
    bool drain = false;  // stores of an epilogue are outstanding: counted waits do not hold

    while (cw < ws.items) {
        const bool wave_live = wm * WTM < cc.rows_in && wn * WTN < cc.cols_in;  // wave-uniform
        v4f acc[TN][TM];
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
        for (int kt = 0; kt < nkt; ++kt) {
            const uint8_t* cur = s_ring + cslot * kStage;
            if (kt % kSclBlocks == 0) cchunk = cchunk + 1 < kSlots ? cchunk + 1 : 0;
            int issued = 0;
            if (!late || !wave_live) issued = produce_issue();
            if (kt == nkt - 1 && K % kSB != 0) {
                // the pieces past the end of K hold other bytes: zero them
                const int good = (int)(K % kSB) / 16;
                uint8_t* z = s_ring + cslot * kStage;
                for (int r = wave * kWave + lane_id<kFresh>(); r < BM + BN; r += NT) {
                    const int row = r < BM ? r : r - BM;
                    for (int p = good; p < 8; ++p)
                        *reinterpret_cast<uint4*>(z + (r < BM ? 0 : kAStage) + swz<kSB>(row, p)) =
                            make_uint4(0, 0, 0, 0);
                }
                __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
                __asm__ volatile("" ::: "memory");
                __builtin_amdgcn_s_barrier();
                __asm__ volatile("" ::: "memory");
            }
            if (wave_live) {
                // fragment addresses inside the slot: row l16 of the wave's first 16, pieces kg and kg + 4
                const int lane = lane_id<kFresh>(), l16 = lane & 15;
                const int fa = (wm * WTM + l16) * kSB, fb = kAStage + (wn * WTN + l16) * kSB;
                const int p0 = swz_chunk<kSB>(l16, lane >> 4) << 4, p1 = p0 ^ 64;
                auto frag = [&](int at) {
                    const uint4 x0 = *reinterpret_cast<const uint4*>(cur + at + p0);
                    const uint4 x1 = *reinterpret_cast<const uint4*>(cur + at + p1);
                    return v8i{(int)x0.x, (int)x0.y, (int)x0.z, (int)x0.w,
                               (int)x1.x, (int)x1.y, (int)x1.z, (int)x1.w};
                };
                const float* scl = reinterpret_cast<const float*>(s_scl + cchunk * kScl) + kt % kSclBlocks;
                v8i tf[TM], nf[2];
                float s[TM];
                nf[0] = frag(fb);
#pragma unroll
                for (int j = 0; j < TM; ++j) tf[j] = frag(fa + j * 16 * kSB);
#pragma unroll
                for (int j = 0; j < TM; ++j) s[j] = scl[(wm * WTM + j * 16 + l16) * kSclBlocks];
                const float sb = scl[kSclA / 4 + (wn * WTN / 128) * kSclBlocks];
                if (TN > 1) nf[1] = frag(fb + 16 * kSB);
                // Step q multiplies column block q / TM by token block q % TM; the
                // product of step q - kLag, out of the matrix core by then, is added.
                constexpr int kSteps = TN * TM, kLag = 3;
                v4f part[kLag + 1];
#pragma unroll
                for (int q = 0; q < kSteps + kLag; ++q) {
                    if (q < kSteps) {
                        const int i = q / TM, j = q % TM;
                        part[q % (kLag + 1)] = mma128(nf[i & 1], tf[j]);
                        __builtin_amdgcn_sched_barrier(0);
                        if (q == kLate && late) issued = produce_issue();
                        if (j == TM - 1 && i + 2 < TN) nf[i & 1] = frag(fb + (i + 2) * 16 * kSB);
                        if (q < TM) s[q] *= sb;
                    }
                    if (q >= kLag) {
                        const int i = (q - kLag) / TM, j = (q - kLag) % TM;
                        const v4f& pt = part[(q - kLag) % (kLag + 1)];
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(pt[r], s[j], acc[i][j][r]);
                    }
                    __builtin_amdgcn_sched_barrier(0);  // keep the steps in this order
                }
            }
            produce_next();
            // the next stage must have landed; those issued after it may stay in flight
            if (kAhead == 1 || drain || issued == 0) stage_barrier<0>();
            else if (issued == L) stage_barrier<L>();
            else stage_barrier<L + S_J + 1>();
            drain = false;
            if (kt + 1 < nkt) cslot = cslot + 1 < kSlots ? cslot + 1 : 0;
        }

        // ---- epilogue.  The slot just consumed is free; the others hold the
        // next tile's first stages.  BF16 rows are staged there, half the tile
        // at a time, 16-byte pieces XOR-swizzled by the row so that the lanes'
        // 8-byte writes (16 rows at one column) and the readers' whole rows are
        // both conflict-free, then written out in 16-byte pieces.
        const int lane = lane_id<kFresh>(), l16 = lane & 15, kg = lane >> 4, tid = wave * kWave + lane;
        uint8_t* stg = s_ring + cslot * kStage;
        if ((args.N & 7) == 0) {
            constexpr int kPasses = BM * BN * 2 > kStage ? 2 : 1;
            constexpr int kRows = BM / kPasses, kPieces = BN / 8;
            static_assert(kRows * BN * 2 <= kStage && TL::WGM % kPasses == 0, "a pass fits the slot");
#pragma unroll
            for (int pass = 0; pass < kPasses; ++pass) {
                if (pass * kRows >= cc.rows_in) break;  // uniform
                if (wave_live && wm / (TL::WGM / kPasses) == pass) {
#pragma unroll
                    for (int j = 0; j < TM; ++j) {
                        const int row = wm * WTM - pass * kRows + j * 16 + l16;
#pragma unroll
                        for (int i = 0; i < TN; ++i) {
                            const int col = wn * WTN + i * 16 + kg * 4;
                            *reinterpret_cast<uint2*>(stg + row * (BN * 2) + (((col / 8) ^ (row & 15)) << 4) +
                                                      (col & 4) * 2) =
                                make_uint2(f32x2_to_bf16x2(acc[i][j][0], acc[i][j][1]),
                                           f32x2_to_bf16x2(acc[i][j][2], acc[i][j][3]));
                        }
                    }
                }
                __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
                __asm__ volatile("" ::: "memory");
                __builtin_amdgcn_s_barrier();
                __asm__ volatile("" ::: "memory");
#pragma unroll 1
                for (int q = tid; q < kRows * kPieces; q += NT) {
                    const int row = q / kPieces, p = q % kPieces;
                    if (pass * kRows + row < cc.rows_in && p * 8 < cc.cols_in)
                        store_stream16(args.c + (cc.m0 + pass * kRows + row) * args.N + cc.n0 + p * 8,
                                       *reinterpret_cast<const uint4*>(stg + row * (BN * 2) + ((p ^ (row & 15)) << 4)));
                }
                // the slot is written again: by the next pass, or by the next stage's loads
                __builtin_amdgcn_s_waitcnt(0xc07f);
                __asm__ volatile("" ::: "memory");
                __builtin_amdgcn_s_barrier();
                __asm__ volatile("" ::: "memory");
            }
        } else if (wave_live) {
            // rows of c that do not start on 16 bytes: element stores
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int row = wm * WTM + j * 16 + l16;
                if (row >= cc.rows_in) continue;
#pragma unroll
                for (int i = 0; i < TN; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int col = wn * WTN + i * 16 + kg * 4 + r;
                        if (col < cc.cols_in)
                            args.c[(cc.m0 + row) * args.N + cc.n0 + col] = (uint16_t)f32_to_bf16(acc[i][j][r]);
                    }
            }
        }
        drain = true;
        cslot = cslot + 1 < kSlots ? cslot + 1 : 0;
        cw += gridDim.x;
        next_item(cw, cc);
    }
}

// ---------------------------------------------------------------------------
// Few rows per group: the weights are read once each and nothing else matters,
// so they go from memory straight into the matrix core's registers.  A
// workgroup's SPLIT waves share NF x 16 columns of one group and take every
// SPLIT-th scale block of K each (together whole stretches of a weight row),
// kDeep blocks ahead; their sums are joined in LDS in wave order.  The grid is
// (columns, groups): no tile map, an empty group's workgroups leave at once, the
// others take the group's first 16 rows.  What lies past them (the host does not see
// the group sizes) goes to `extra` more workgroups a column, first in the grid since
// theirs is the longest way: 1024 rows of 256 groups, 2048 x 1024, all in one group
// 36 us instead of 240 with a group's workgroups looping over its rows; even groups
// 95 instead of 92.
// A lane's operand pieces are 64 bytes apart (pieces kg and kg + 4 of a block),
// so the four lanes of a row read 64 bytes together; with the nontemporal hint
// the two halves of a line were fetched twice (K 7168, N 2048, 8 rows of 64
// experts: a quarter more time).  Measured there, 8 rows: 25 us (4.6 TB/s of
// weights; the 32 x 128 tile 36); 64 rows, a few a group: 105 us (120), and on the
// same rows one 16-column fragment a wave instead of two 1 % more, eight waves
// instead of four 50 %, eight blocks ahead instead of four 23 %, two row blocks of
// 16 instead of one 25 %.
template <int NF, int SPLIT>
__global__ __launch_bounds__(SPLIT * kWave, 1) void block128_rows_kernel(const GemmArgs args) {
    constexpr int kDeep = 4, kCols = NF * 16, kRows = 16, NT = SPLIT * kWave;
    __shared__ float s_sum[SPLIT][kRows][kCols + 1];
    __shared__ uint32_t s_wave[SPLIT];
    __shared__ int s_group, s_block;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), l16 = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int64_t K = args.K, N = args.N, n0 = (int64_t)blockIdx.x * kCols;
    const int nkt = (int)((K + kSB - 1) / kSB);
    const int mine = (nkt - wave + SPLIT - 1) / SPLIT;  // blocks wave, wave + SPLIT, ...

    // rows m0 .. m0 + 15 below hi, of expert e
    auto rows16 = [&](int e, int64_t m0, int64_t hi) {
        const uint8_t* bp[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const int64_t n = n0 + f * 16 + l16;
            bp[f] = args.b + ((int64_t)e * N + (n < N ? n : N - 1)) * K;  // columns past N re-read the last
        }
        const float* bs = static_cast<const float*>(args.bs) + ((int64_t)e * ((N + 127) / 128) + n0 / 128) * nkt;
        const int rows_in = (int)(hi - m0 < kRows ? hi - m0 : kRows);
        const int64_t r = m0 + (l16 < rows_in ? l16 : rows_in - 1);  // rows past the group re-read its last
        const uint8_t* ap = args.a + r * K;
        const float* sp = static_cast<const float*>(args.as) + r * nkt;
        uint4 wb[kDeep][NF][2], ta[kDeep][2];
        float sa[kDeep], sb[kDeep];
        // block i of this wave into buffer d; TAIL: it may be the shorter last one
        auto load = [&](int i, int d, auto tail) {
            const int kb = wave + i * SPLIT;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int64_t at = (int64_t)kb * kSB + (kg + 4 * c) * 16;
                const bool in = !tail || at < K;
#pragma unroll
                for (int f = 0; f < NF; ++f)
                    wb[d][f][c] = in ? *reinterpret_cast<const uint4*>(bp[f] + at) : make_uint4(0, 0, 0, 0);
                ta[d][c] = in ? *reinterpret_cast<const uint4*>(ap + at) : make_uint4(0, 0, 0, 0);
            }
            sa[d] = sp[kb];
            sb[d] = bs[kb];
        };
        v4f acc[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f) acc[f] = v4f{0.f, 0.f, 0.f, 0.f};
        auto frag = [](const uint4 (&x)[2]) {
            return v8i{(int)x[0].x, (int)x[0].y, (int)x[0].z, (int)x[0].w,
                       (int)x[1].x, (int)x[1].y, (int)x[1].z, (int)x[1].w};
        };
        auto add = [&](int d) {
            const float s = sa[d] * sb[d];
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const v4f p = mma128(frag(wb[d][f]), frag(ta[d]));
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[f][j] = fmaf(p[j], s, acc[f][j]);
            }
        };
        // whole rounds of kDeep blocks keep kDeep - 1 loads in flight without a
        // branch; the last two rounds check each block
        constexpr std::true_type kTail{};
        constexpr std::false_type kWhole{};
        const int rounds = K % kSB == 0 ? mine / kDeep : (mine - 1) / kDeep;  // of blocks that are whole
        int i = 0;
        if (rounds > 0) {
#pragma unroll
            for (int d = 0; d < kDeep; ++d) load(d, d, kWhole);
            for (i = 0; i + kDeep < rounds * kDeep; i += kDeep) {
#pragma unroll
                for (int d = 0; d < kDeep; ++d) {
                    add(d);
                    load(i + kDeep + d, d, kWhole);
                }
            }
#pragma unroll
            for (int d = 0; d < kDeep; ++d) {
                add(d);
                if (i + kDeep + d < mine) load(i + kDeep + d, d, kTail);
            }
            i += kDeep;
        } else {
#pragma unroll
            for (int d = 0; d < kDeep; ++d)
                if (d < mine) load(d, d, kTail);
        }
#pragma unroll
        for (int d = 0; d < kDeep; ++d)
            if (i + d < mine) add(d);
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int j = 0; j < 4; ++j) s_sum[wave][l16][f * 16 + kg * 4 + j] = acc[f][j];
        __syncthreads();
        for (int q = tid; q < rows_in * kCols; q += NT) {
            const int row = q / kCols, col = q % kCols;
            float v = s_sum[0][row][col];
#pragma unroll
            for (int w = 1; w < SPLIT; ++w) v += s_sum[w][row][col];
            if (n0 + col < N) args.c[(m0 + row) * N + n0 + col] = (uint16_t)f32_to_bf16(v);
        }
        __syncthreads();  // the sums are written again for the next rows
    };

    const int G = args.G, extra = (int)gridDim.y - G;  // extra 0: each group's workgroups take all of its rows
    if ((int)blockIdx.y >= extra) {
        const int g = (int)blockIdx.y - extra;
        const GroupRange gr = group_range(args.off, args.ids, g, args.T, args.E);
        if (gr.hi <= gr.lo) return;  // workgroup-uniform
        const int e = args.ids[g];
        int64_t m0 = gr.lo;
        do rows16(e, m0, gr.hi);
        while (extra == 0 && (m0 += kRows) < gr.hi);
        return;
    }
    // The blocks of 16 rows past each group's first: the q-th of all of them, by a sum
    // over the groups' numbers of them, kGroups consecutive groups a thread.
    constexpr int kGroups = kMaxGroups / NT;
    uint32_t blocks[kGroups], sum = 0;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int g = tid * kGroups + i;
        blocks[i] = 0;
        if (g < G) {
            const GroupRange gr = group_range(args.off, args.ids, g, args.T, args.E);
            if (gr.hi > gr.lo) blocks[i] = (uint32_t)((gr.hi - gr.lo - 1) / kRows);
        }
        sum += blocks[i];
    }
    uint32_t total;
    const uint32_t before = block_exclusive_scan<NT>(sum, s_wave, &total);
    for (uint32_t q = blockIdx.y; q < total; q += extra) {
        uint32_t at = before;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            if (q >= at && q - at < blocks[i]) {
                s_group = tid * kGroups + i;
                s_block = (int)(q - at) + 1;
            }
            at += blocks[i];
        }
        __syncthreads();
        const int g = __builtin_amdgcn_readfirstlane(s_group);
        const int64_t block = __builtin_amdgcn_readfirstlane(s_block);
        const GroupRange gr = group_range(args.off, args.ids, g, args.T, args.E);
        rows16(args.ids[g], gr.lo + block * kRows, gr.hi);  // ends with a barrier: s_group may be written again
    }
}

int64_t compute_units() {
    const int cus = device_cus();
    return cus > 0 ? cus : 256;
}

constexpr int kRowFrags = 2, kRowCols = kRowFrags * 16, kRowSplit = 4;

hipError_t launch_rows(const GemmProblem& p, int64_t cus, hipStream_t stream) {
    int64_t grid = 0;
    const GemmArgs a = make_args(p, 16, kRowCols, 1, 1, &grid);
    // the first rows of the grid take what lies past 16 rows in a group: as many as
    // fill the chip, fewer where T holds fewer blocks
    const int64_t fill = (2 * cus + a.ntiles_n - 1) / a.ntiles_n, extra = p.T / 16 < fill ? p.T / 16 : fill;
    const dim3 blocks((unsigned)a.ntiles_n, (unsigned)(p.G + extra));
    hipLaunchKernelGGL((block128_rows_kernel<kRowFrags, kRowSplit>), blocks, dim3(kRowSplit * kWave), 0, stream, a);
    return hipGetLastError();
}

template <class TL>
hipError_t launch_tile(const GemmProblem& p, hipStream_t stream, int mband) {
    int64_t grid = 0;
    const GemmArgs a = make_args(p, TL::BM, TL::BN, mband, 1, &grid);  // one workgroup per CU: the ring fills its LDS
    if (grid <= 0) return hipSuccess;
    hipLaunchKernelGGL(block128_kernel<TL>, dim3((unsigned)grid), dim3(TL::kThreads), 0, stream, a);
    return hipGetLastError();
}

using TileLarge = BTile<256, 256, 4, 2, 2, 8>;
using TileMid = BTile<128, 256, 2, 4, 3, 4>;
using TileSmall = BTile<32, 128, 1, 4, 4, 8>;

}  // namespace

int block128_tile_choice(const GemmProblem& p) {
    const int64_t cus = compute_units();
    const int64_t groups = p.G < p.T ? p.G : p.T;
    if (groups <= 0) return 0;
    // Rows per group: the average, moved halfway to the host's hint of the largest.
    const int64_t avg = p.T / groups;
    const int64_t hint = p.max_rows_hint < p.T ? p.max_rows_hint : p.T;
    const int64_t rows = hint > avg ? (avg + hint) / 2 : avg;
    // Rounds of a persistent launch over BM x BN tiles.  The host does not see
    // the group sizes: T / BM whole tiles and a partial one, half a tile on
    // average, per group; at least a tile for each.
    auto rounds = [&](int64_t BM, int64_t BN) {
        const int64_t half = (2 * p.T + groups * BM) / (2 * BM), mt = half > groups ? half : groups;
        return (mt * ((p.N + BN - 1) / BN) + cus - 1) / cus;
    };
    // A round of 256 x 256 tiles takes 66 us at K = 4096, of 128 x 256 tiles 44,
    // of 32 x 128 tiles 20 to 25; the fewest weighted rounds win.  Measured on
    // operands that no cache holds (us, 256 / 128 / 32 rows a tile): 65536 rows of
    // 128 uneven experts, 4096 x 1536: 500 / 602 / 1826; 5003 of 24, 2080 x 1000:
    // 51 / 34 / 73; 4096 of 64, 4096 x 2048: 153 / 108 / 197; 256 of 4, 4096 x
    // 2048: - / 38 / 23; 400 of 2: - / 38 / 23.
    const int64_t c256 = 66 * rounds(256, 256), c128 = 44 * rounds(128, 256), c32 = 24 * rounds(32, 128);
    // The row kernel reads an expert's weights once per 16 rows: 2 rows a group
    // 133 us against 147 for the tiles, 4 rows 159 against 164, 8 rows 177 against
    // 168 (64 experts, 7168 x 2048).  One long group among short ones: 512 rows of
    // 128, 146 in the longest, 4096 x 1536, 121 against 123; 1024 of 256, 256 in it,
    // 2048 x 1024, 73 against 63.
    // Where the 32 x 128 tiles do not fill the chip it still wins at 8 rows (8
    // experts, 2048 x 1024: 10.6 us against 14.5).
    const bool wide_grid = (p.N + kRowCols - 1) / kRowCols * p.G < (1 << 22);
    const bool few = avg <= 4 && hint <= 128, small = rows <= 16 && (p.N + 127) / 128 * groups < cus;
    if (wide_grid && (few || small)) return 16;
    if (c32 < c128 && c32 < c256) return 32;
    return c128 <= c256 ? 128 : 256;
}

hipError_t launch_grouped_gemm_block128(const GemmProblem& p, hipStream_t stream) {
    switch (block128_tile_choice(p)) {
        case 16: return launch_rows(p, compute_units(), stream);
        case 32: return launch_tile<TileSmall>(p, stream, 1 << 30);
        case 128: return launch_tile<TileMid>(p, stream, 4);
        case 256: return launch_tile<TileLarge>(p, stream, 4);
        default: return hipSuccess;  // no groups or no rows
    }
}

}  // namespace mxg
