// gemm_bf16_tile.h -- the K pipeline of the BF16 products: operand stages of 64 in
// depth through a ring of LDS slots filled by direct global->LDS loads, read into the
// matrix core's registers one step ahead.  Device code for gfx950.
//
//  * Matrix core: v_mfma_f32_16x16x32_bf16, accumulating.  Operands trade places as in
//    the FP8 products: the operand whose rows become the output's columns is the
//    instruction's A, so a lane's four results are four neighbouring columns of a row.
//  * An operand is either deep (its rows run along the depth: stage rows of 128 bytes,
//    16-byte pieces XOR-swizzled, read 16 bytes a lane) or wide (the depth is its row
//    index: stage rows of R elements, 32-byte pieces XOR-swizzled, read through the
//    transposing LDS load, which gives a lane four depths of its column).
//  * Loads go through buffer descriptors whose range ends behind the tile's rows (or its
//    depth); a lane whose piece lies past the columns (or the depth) asks for an offset
//    past every range.  What is past the range reads nothing and leaves zeros in LDS, so
//    rows and tails of any size need no second path, and what lies behind them (another
//    expert's rows, whatever they hold) takes no part.
//  * A stage is two steps of 32 in depth.  While a step is multiplied, the next step's
//    fragments replace its own, one by one.  Two barriers a stage: behind the first
//    (all waves have read the slot) its slot is filled with the stage that follows those
//    in the ring; behind the second (the next stage has landed) the next stage's fragments
//    are read.  The stages run on across tiles: an epilogue has the next tile's first
//    stages in flight behind it.
//  * Slots: a stage of 256 x 256 takes 1.4 us, longer than its loads, so two slots (128 KB)
//    do.  A stage of 128 x 128 takes 0.4 us, a load up to 1.2: four slots of half the size
//    (2048^3: 24 us against 43 with two and two workgroups a CU); 64 x 128 five, 32 x 128 six.
#pragma once

#include "gemm_bf16.h"
#include "gemm_common.h"

namespace mxg {
namespace bf16 {

using gemm::stage_barrier;
using gemm::swz_chunk;

constexpr int kStageDepth = 64;
constexpr uint32_t kNowhere = 0x80000000u;  // an offset past every descriptor's range

typedef int v4i __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));

// Direct-to-LDS loads of 16 bytes a lane (lane l to lds + 16 l; the next load's 1 KiB follow) at off + soff from a
// buffer descriptor's base; all but off in scalar registers.  The wait states stand here, since nothing outside
// keeps its place before an assembly load and the compiler gives it none: five (s_mov and s_nop 3) between a vector
// instruction's write of a scalar register and the load that reads it -- a lane read that makes the descriptor, or
// one that brings back a spilled offset -- and one behind each write of M0.  Loads that follow each other share them
// (1 x 4096 of 4096, 16 x 32 split: 8.8 us with five states each, 8.1 so).
__device__ __forceinline__ void lds_load(const v4i& desc, uint32_t off, uint32_t soff, uint32_t lds) {
    __asm__ volatile(
        "s_mov_b32 m0, %3\n\ts_nop 3\n\t"
        "buffer_load_dwordx4 %0, %1, %2 offen lds"
        :
        : "v"(off), "s"(desc), "s"(soff), "s"(lds)
        : "memory", "m0");
}
__device__ __forceinline__ void lds_load2(const v4i& desc, uint32_t off0, uint32_t off1, uint32_t soff0, uint32_t soff1,
                                          uint32_t lds) {
    __asm__ volatile(
        "s_mov_b32 m0, %5\n\ts_nop 3\n\t"
        "buffer_load_dwordx4 %0, %2, %3 offen lds\n\ts_add_u32 m0, m0, 1024\n\ts_nop 0\n\t"
        "buffer_load_dwordx4 %1, %2, %4 offen lds"
        :
        : "v"(off0), "v"(off1), "s"(desc), "s"(soff0), "s"(soff1), "s"(lds)
        : "memory", "m0", "scc");
}
__device__ __forceinline__ void lds_load4(const v4i& desc, uint32_t off0, uint32_t off1, uint32_t off2, uint32_t off3,
                                          uint32_t soff0, uint32_t soff1, uint32_t soff2, uint32_t soff3, uint32_t lds) {
    __asm__ volatile(
        "s_mov_b32 m0, %9\n\ts_nop 3\n\t"
        "buffer_load_dwordx4 %0, %4, %5 offen lds\n\ts_add_u32 m0, m0, 1024\n\ts_nop 0\n\t"
        "buffer_load_dwordx4 %1, %4, %6 offen lds\n\ts_add_u32 m0, m0, 1024\n\ts_nop 0\n\t"
        "buffer_load_dwordx4 %2, %4, %7 offen lds\n\ts_add_u32 m0, m0, 1024\n\ts_nop 0\n\t"
        "buffer_load_dwordx4 %3, %4, %8 offen lds"
        :
        : "v"(off0), "v"(off1), "v"(off2), "v"(off3), "s"(desc), "s"(soff0), "s"(soff1), "s"(soff2), "s"(soff3), "s"(lds)
        : "memory", "m0", "scc");
}

// One operand's stage: R rows of the output (or its columns), NW waves filling it.
template <int R, bool WIDE, int NW>
struct Operand {
    static constexpr int kBytes = R * kStageDepth * 2;
    static constexpr int kLoads = kBytes / 1024 / NW;            // a wave's
    static constexpr int kRowBytes = WIDE ? R * 2 : 128;
    static constexpr int kLanes = kRowBytes / 16;                // lanes a stage row
    static constexpr int kRows = 64 / kLanes;                    // stage rows a load
    static_assert(kLoads * NW * 1024 == kBytes, "whole loads");
    static_assert(!WIDE || R >= 32, "a wide stage row holds two pieces of 32 bytes at least");

    // Wide rows: the 32-byte pieces of a row are XORed with this, so that the eight rows
    // that half a wave reads at one column ({0..3} and {8..11} beside a multiple of 4)
    // lie in distinct banks.  Rows of 128 and 64 bytes already differ by their address.
    static __device__ __forceinline__ int turn(int row) {
        constexpr int kPieces = kRowBytes / 32;
        if constexpr (kPieces >= 8) return (row & 3) | ((row >> 3) & 1) << 2;
        else if constexpr (kPieces == 4) return ((row >> 1) & 1) | ((row >> 3) & 1) << 1;
        else return (row >> 3) & 1;
    }

    static constexpr bool kWide = WIDE;
    static constexpr int kStep = NW * kRows;                     // stage rows from a load to a wave's next
    // the swizzles repeat every 16 rows: so many of a wave's loads differ by more than their row
    static constexpr int kOffs = kStep % 16 == 0 ? 1 : kStep % 8 == 0 ? 2 : 4;
    static_assert(kStep % 4 == 0 && (kLoads % kOffs == 0 || kLoads < kOffs), "whole turns of the swizzle");
    uint32_t off[kOffs];

    static __device__ __forceinline__ int stage_row(int wave, int lane, int j) {
        return (wave + NW * j) * kRows + lane / kLanes;
    }
    // which 16-byte piece of the source row this lane fetches
    static __device__ __forceinline__ int piece(int row, int lane) {
        if constexpr (WIDE) return (lane % kLanes) ^ (turn(row) << 1);
        else return swz_chunk<128>(row, lane % 8);
    }
    // This lane's offsets in a tile of `real` columns (wide), in a stage with `left` of the depth before it
    // (deep: its pieces past the end ask for what lies past the range).
    __device__ __forceinline__ void set(int wave, int lane, int real, int left, uint32_t ld) {
#pragma unroll
        for (int j = 0; j < kOffs; ++j) {
            const int row = stage_row(wave, lane, j), p = piece(row, lane);
            off[j] = p * 8 < (WIDE ? real : left) ? (uint32_t)row * ld + p * 16 : kNowhere;
        }
    }
    // The descriptor's range, from the stage's base: it ends behind the tile's last row (deep: behind the
    // end of that row, `left` of whose depth lies before it), or behind the depth's last row (wide).
    static __device__ __forceinline__ int range(int real, int left, int depth, uint32_t ld) {
        if constexpr (WIDE) return (left < kStageDepth ? left : kStageDepth) * (int)ld;
        else return (int)((uint32_t)real * ld - (uint32_t)(depth - left) * 2);
    }
    __device__ __forceinline__ void load(const v4i& desc, int j, uint32_t ld, uint32_t lds) const {
        lds_load(desc, off[j % kOffs], soff(j, ld), lds + j * (NW * 1024));
    }
    static __device__ __forceinline__ uint32_t soff(int j, uint32_t ld) {
        return (uint32_t)(j / kOffs * kOffs * kStep) * ld;
    }
    // All of the stage, by one wave.
    __device__ __forceinline__ void load_all(const v4i& desc, uint32_t ld, uint32_t lds) const {
        static_assert(NW == 1 && (kLoads == 2 || kLoads % 4 == 0), "loads in twos or fours, 1 KiB apart");
        if constexpr (kLoads == 2) {
            lds_load2(desc, off[0], off[1 % kOffs], soff(0, ld), soff(1, ld), lds);
        } else {
#pragma unroll
            for (int j = 0; j < kLoads; j += 4)
                lds_load4(desc, off[j % kOffs], off[(j + 1) % kOffs], off[(j + 2) % kOffs], off[(j + 3) % kOffs],
                          soff(j, ld), soff(j + 1, ld), soff(j + 2, ld), soff(j + 3, ld), lds + j * 1024);
        }
    }
    // bytes the base moves a stage
    static __device__ __forceinline__ int64_t step(int64_t ld) { return WIDE ? kStageDepth * ld : 128; }

    // This lane's part of the addresses of the fragments from the first-th on (of 16 rows each; first a
    // multiple of how many there are).
    static __device__ __forceinline__ uint32_t lane_base(int lane, int first) {
        const int l16 = lane & 15, kg = lane >> 4;
        if constexpr (WIDE) {
            const int row = kg * 8 + l16 / 4;
            return row * kRowBytes + ((turn(row) ^ first) << 5) + (l16 & 3) * 8;
        } else {
            return (first * 16 + l16) * 128 + (swz_chunk<128>(l16, kg) << 4);
        }
    }
    // The f-th of them, step (0 or 1); at: lane_base and the stage's LDS address, whose low 9 bits are 0.
    static __device__ __forceinline__ v8b frag(uint32_t at, int f, int step) {
        if constexpr (WIDE) {
            typedef v4s __attribute__((address_space(3)))* lp;
            const uint32_t p = (at ^ (f << 5)) + step * 32 * kRowBytes;
            union {
                v4s s[2];
                v8b b;
            } u;
            u.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(size_t)p);
            u.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(size_t)(p + 4 * kRowBytes));
            return u.b;
        } else {
            typedef const v8b __attribute__((address_space(3)))* lp;
            return *(lp)(size_t)((at ^ (step << 6)) + f * (16 * 128));
        }
    }
};

// A tile of BM x BN outputs by WGM x WGN waves; A gives the rows, B the columns.
template <int BM_, int BN_, int WGM_, int WGN_, int SLOTS_, bool AWIDE_, bool BWIDE_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_;
    static constexpr int kSlots = SLOTS_;  // stages in LDS
    static constexpr bool AWIDE = AWIDE_, BWIDE = BWIDE_;
    static constexpr int kWaves = WGM * WGN, kThreads = kWave * kWaves;
    static constexpr int TM = BM / WGM / 16, TN = BN / WGN / 16;  // fragments a wave
    using A = Operand<BM, AWIDE, kWaves>;
    using B = Operand<BN, BWIDE, kWaves>;
    static constexpr int kStage = A::kBytes + B::kBytes;
    static constexpr int kLoads = A::kLoads + B::kLoads;
    static constexpr int kOut = 2048;  // bytes of LDS a wave's epilogue passes its results through
    static constexpr int kRing = kSlots * kStage, kLds = kRing + kWaves * kOut;
    // column blocks of a stage's second step behind which the two barriers stand
    static constexpr int kRead = TN >= 8 ? 1 : 0, kLanded = TN >= 8 ? 3 : TN >= 4 ? 1 : TN - 1;
    // A stage's loads are spread over the column blocks from kRead on, about one a block: the loads'
    // path moves 64 bytes a cycle, and waves that issue faster wait.  How many stand before block i:
    static constexpr int loads_before(int i) { return kLoads * (i - kRead) / (TN - kRead); }
};

// Work items of a persistent launch of `grid` workgroups: whole tiles, but where the last round is at
// most half full, each of its tiles is two items of half its columns.
struct Items {
    int full, all;  // items that are whole tiles; all of them
};
__device__ __forceinline__ Items items_of(int tiles, int grid) {
    const int rest = tiles % grid;
    return rest > 0 && 2 * rest <= grid ? Items{tiles - rest, tiles + rest} : Items{tiles, tiles};
}

// The sum of a fragment's 8 values in this lane's row.
__device__ __forceinline__ float frag_sum(const v8b& f) {
    union {
        v8b b;
        uint32_t w[4];
    } u;
    u.b = f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) s += __uint_as_float(u.w[i] << 16) + __uint_as_float(u.w[i] & 0xffff0000u);
    return s;
}

// The lane number, made anew where it is needed: what derives from it holds no register
// between stages.
__device__ __forceinline__ int fresh_lane() {
    int l;
    __asm__ volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(l));
    return l;
}

// Runs the tiles of `job`.  Job:
//   Coord        int rows_in, cols_in, stages (of the whole tile), depth (of the present segment);
//                const uint8_t *a, *b (that segment's first stage)
//   bool next(int& W, Coord&)       the first item from W on that there is, or false
//   bool segment(Coord&)            the tile's next stretch of depth, or false
//   lda, ldb                        bytes a row of the operands
//   void finish(c, acc, wm, wn, out)   epilogue of a wave's accumulators
//   kSums, bool sums(c), void put_sum(c, row, v)   whether A's rows are added up over the depth
//                beside the product, in which tiles, and where a sum goes
template <class TL, class Job>
__device__ __forceinline__ void run_tiles(Job& job, uint8_t* s_ring, int first, int step) {
    constexpr int TM = TL::TM, TN = TL::TN;
    using A = typename TL::A;
    using B = typename TL::B;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / TL::WGN, wn = wave % TL::WGN;

    typename Job::Coord cc{};
    int cw = first;
    if (!job.next(cw, cc)) return;  // workgroup-uniform

    // ---- the producer: kSlots stages ahead.  Pointers, ranges, offsets and `left` (depth from its stage to
    // the segment's end) are those of its next stage; past the last tile `left` is 0 and its loads
    // have an empty range, so that they need no branch.
    typename Job::Coord pc = cc;
    int pw = cw, left = 0, ra = 0, rb = 0;  // ra, rb: the ranges
    uint64_t pa = 0, pb = 0;
    const uint32_t slot0 = (uint32_t)__builtin_amdgcn_readfirstlane(gemm::lds_addr(s_ring) + wave * 1024);
    uint32_t slot = slot0;
    const int64_t sa = gemm::first_lane64(A::step(job.lda)), sb = gemm::first_lane64(B::step(job.ldb));
    A fa;
    B fb;
    const uint32_t lda = (uint32_t)job.lda, ldb = (uint32_t)job.ldb;
    auto offsets = [&]() {
        const int lane = fresh_lane();
        fa.set(wave, lane, pc.rows_in, left, lda);
        fb.set(wave, lane, pc.cols_in, left, ldb);
        ra = __builtin_amdgcn_readfirstlane(A::range(pc.rows_in, left, pc.depth, lda));
        rb = __builtin_amdgcn_readfirstlane(B::range(pc.cols_in, left, pc.depth, ldb));
    };
    auto begin = [&]() {  // the first stage of pc's segment
        pa = (uint64_t)gemm::first_lane64((int64_t)pc.a);
        pb = (uint64_t)gemm::first_lane64((int64_t)pc.b);
        left = __builtin_amdgcn_readfirstlane(pc.depth);
        offsets();
    };
    auto next_tile = [&](bool more) {
        while (more && pc.stages == 0) {
            pw += step;
            more = job.next(pw, pc);
        }
        if (more) begin();
        else left = ra = rb = 0;
    };
    struct Where {
        v4i da, db;
        uint32_t slot;
    };
    auto where = [&]() {
        // (scalar already; the lane reads say so where the compiler cannot tell)
        const uint64_t ua = (uint64_t)gemm::first_lane64((int64_t)pa), ub = (uint64_t)gemm::first_lane64((int64_t)pb);
        return Where{{(int)(uint32_t)ua, (int)(uint32_t)(ua >> 32), __builtin_amdgcn_readfirstlane(ra), 0x00020000},
                     {(int)(uint32_t)ub, (int)(uint32_t)(ub >> 32), __builtin_amdgcn_readfirstlane(rb), 0x00020000},
                     (uint32_t)__builtin_amdgcn_readfirstlane(slot)};
    };
    auto load = [&](const Where& w, int l) {
        if (l < A::kLoads) fa.load(w.da, l, lda, w.slot);
        else fb.load(w.db, l - A::kLoads, ldb, w.slot + A::kBytes);
    };
    auto load_all = [&]() {
        const Where w = where();
#pragma unroll
        for (int l = 0; l < TL::kLoads; ++l) load(w, l);
    };
    auto advance = [&]() {  // behind a stage's loads
        if constexpr (TL::kSlots == 2) slot = 2 * slot0 + TL::kStage - slot;
        else slot = slot < slot0 + TL::kRing - TL::kStage ? slot + TL::kStage : slot0;
        pa += sa;
        pb += sb;
        if (left == 0) return;  // past the last tile
        left -= kStageDepth;
        if (!A::kWide) ra -= kStageDepth * 2;
        if (!B::kWide) rb -= kStageDepth * 2;
        if (left < kStageDepth) {
            if (left > 0) offsets();  // a last stage that is not whole
            else if (job.segment(pc)) begin();
            else {
                pw += step;
                next_tile(job.next(pw, pc));
            }
        }
    };
    next_tile(true);
#pragma unroll
    for (int i = 0; i < TL::kSlots; ++i) {
        load_all();
        advance();
    }
    stage_barrier<(TL::kSlots - 1) * TL::kLoads>();

    // ---- the consumer
    v8b tf[2][TM], nf[TN];
    uint32_t abase, bbase;
    {
        const int lane = threadIdx.x & (kWave - 1);
        abase = A::lane_base(lane, wm * TM);
        bbase = B::lane_base(lane, wn * TN);
    }
    // this lane's addresses in the present stage and in the next (a wide operand's opaque, so that its
    // fragments' own addresses are made where they are read and hold no registers)
    uint32_t ca = gemm::lds_addr(s_ring) + abase, cb = gemm::lds_addr(s_ring) + A::kBytes + bbase;
    const uint32_t turn_a = 2 * ca + TL::kStage, turn_b = 2 * cb + TL::kStage;
    int turn = 0;  // the present slot, where there are more than two
    auto next_slot = [&](uint32_t& na, uint32_t& nb) {
        if constexpr (TL::kSlots == 2) {
            na = turn_a - ca;
            nb = turn_b - cb;
        } else {
            const int by = turn + 1 < TL::kSlots ? TL::kStage : TL::kStage - TL::kRing;
            turn = turn + 1 < TL::kSlots ? turn + 1 : 0;
            na = ca + by;
            nb = cb + by;
        }
    };
    // a stage begins with these fragments in registers, read in this order; the rest follow in it
    constexpr int kPre = TN < 3 ? TN : 3;
    auto first_frags = [&]() {
        nf[0] = B::frag(cb, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            tf[0][j] = A::frag(ca, j, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 1; i < kPre; ++i) {
            nf[i] = B::frag(cb, i, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    bool ahead = false;  // the next stage has landed already
    for (;;) {
        const bool live = wm * TM * 16 < cc.rows_in && wn * TN * 16 < cc.cols_in;  // wave-uniform
        v4f acc[TN][TM];
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
        const int stages = __builtin_amdgcn_readfirstlane(cc.stages);
        float sum[Job::kSums ? TM : 1] = {};
        bool add_up = false;
        if constexpr (Job::kSums) add_up = wn == 0 && job.sums(cc);
        auto read_barrier = [&]() {
            __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's fragments are in registers
            __asm__ volatile("" ::: "memory");
            __builtin_amdgcn_s_barrier();
            __asm__ volatile("" ::: "memory");
        };
        if (live) {
            first_frags();  // (read at the end of the tile before, too: they hold no registers through its epilogue)
            for (int kt = 0; kt < stages; ++kt) {
                const Where w = where();
                uint32_t na, nb;
                next_slot(na, nb);
                if constexpr (A::kWide) __asm__ volatile("" : "+v"(ca), "+v"(na));
                if constexpr (B::kWide) __asm__ volatile("" : "+v"(cb), "+v"(nb));
#pragma unroll
                for (int i = 0; i < TN; ++i) {
#pragma unroll
                    for (int j = 0; j < TM; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(nf[i], tf[0][j], acc[i][j], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    if (i + kPre < TN) nf[i + kPre] = B::frag(cb, i + kPre, 0);
                    nf[i] = B::frag(cb, i, 1);
#pragma unroll
                    for (int j = i * TM / TN; j < (i + 1) * TM / TN; ++j) tf[1][j] = A::frag(ca, j, 1);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if constexpr (Job::kSums)
                    if (add_up)
#pragma unroll
                        for (int j = 0; j < TM; ++j) sum[j] += frag_sum(tf[0][j]) + frag_sum(tf[1][j]);
#pragma unroll
                for (int i = 0; i < TN; ++i) {
#pragma unroll
                    for (int j = 0; j < TM; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(nf[i], tf[1][j], acc[i][j], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    if (i == TL::kRead) read_barrier();
                    if (i >= TL::kRead)
#pragma unroll
                        for (int q = TL::loads_before(i); q < TL::loads_before(i + 1); ++q) load(w, q);
                    if (i == TL::kLanded) {
                        if (!ahead) gemm::wait_vmem<(TL::kSlots - 2) * TL::kLoads + TL::loads_before(TL::kLanded + 1)>();
                        ahead = false;
                        read_barrier();
                    }
                    if (i >= TL::kLanded) {
                        // the next stage's first fragments (nf[0], tf, nf[1] ...), over the blocks left
                        constexpr int kAll = TM + kPre, kLeft = TN - TL::kLanded;
#pragma unroll
                        for (int q = (i - TL::kLanded) * kAll / kLeft; q < (i - TL::kLanded + 1) * kAll / kLeft; ++q) {
                            if (q == 0) nf[0] = B::frag(nb, 0, 0);
                            else if (q <= TM) tf[0][q > 0 && q <= TM ? q - 1 : 0] = A::frag(na, q - 1, 0);
                            else nf[q > TM ? q - TM : 0] = B::frag(nb, q - TM, 0);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                advance();
                ca = na;
                cb = nb;
            }
            // The next tile's stages are awaited here, before the epilogue's stores: behind them its
            // wait would be theirs too.
            gemm::wait_vmem<0>();
            ahead = true;
            job.template finish<TL>(cc, acc, wm, wn, s_ring + TL::kRing + wave * TL::kOut);
            if constexpr (Job::kSums)
                if (add_up)
#pragma unroll
                    for (int j = 0; j < TM; ++j) {
                        float v = sum[j];  // four lanes a row
                        v += __shfl_xor(v, 16, kWave);
                        v += __shfl_xor(v, 32, kWave);
                        const int lane = fresh_lane(), row = (wm * TM + j) * 16 + (lane & 15);
                        if (lane < 16 && row < cc.rows_in) job.put_sum(cc, row, v);
                    }
        } else if (stages > 0) {
            for (int kt = 0; kt < stages; ++kt) {
                read_barrier();
                load_all();
                stage_barrier<(TL::kSlots - 1) * TL::kLoads>();
                ahead = false;
                advance();
                next_slot(ca, cb);
            }
        }
        cw += step;
        if (!job.next(cw, cc)) break;
    }
    gemm::wait_vmem<0>();  // no load may land once the workgroup's LDS belongs to another
}

// A wave's accumulators through its LDS buffer, 8 rows x 64 columns at a time (16 x 32 where the
// wave has fewer columns): put(row, col, v, x) gets 8 neighbouring columns of a row of the tile
// and what fetch(row, col, x) asked for a block before, so that a row of bf16 goes out in whole
// lines of 128 bytes.  LDS serves a wave in order: a block's writes need not wait for the reads
// of the one before.
template <class TL, class X, class Fetch, class Put>
__device__ __forceinline__ void put_rows(const v4f (&acc)[TL::TN][TL::TM], int wm, int wn, int rows, int cols,
                                         uint8_t* out, Fetch fetch, Put put) {
    constexpr int TM = TL::TM, TN = TL::TN;
    constexpr int kFrags = TN % 4 == 0 ? 4 : 2, kRows = 32 / kFrags, kLanes = kFrags * 2;  // lanes a row
    constexpr int kHalves = 16 / kRows, kAcross = TN / kFrags, kBlocks = TM * kHalves * kAcross;
    static_assert(TN % 2 == 0, "column blocks in pairs");
    const int lane = fresh_lane(), l16 = lane & 15, kg = lane >> 4;
    const int r = lane / kLanes, c = lane % kLanes;
    const int row0 = wm * TM * 16 + r, col0 = wn * TN * 16 + c * 8;
    // 16-byte pieces of a row: XORed so that a 16-lane slice of a write (four rows, or more, by four
    // pieces) and of a read (every other piece of two rows or more) lies in distinct banks
    auto at = [&](int row, int piece) -> uint8_t* {
        const int turn = kFrags == 4 ? (row & 3) << 2 | (row & 1) : (row >> 1) & 7;
        return out + row * (kFrags * 64) + ((piece ^ turn) << 4);
    };
    X x[2];
    auto place = [&](int q, int& row, int& col) {  // halves of 16 rows innermost, then across
        row = row0 + q / (kHalves * kAcross) * 16 + q % kHalves * kRows;
        col = col0 + q / kHalves % kAcross * (kFrags * 16);
    };
    auto ask = [&](int q) {
        int row, col;
        place(q, row, col);
        if (row < rows && col < cols) fetch(row, col, x[q & 1]);
    };
    ask(0);
#pragma unroll
    for (int q = 0; q < kBlocks; ++q) {
        const int j = q / (kHalves * kAcross), i = q / kHalves % kAcross * kFrags;
        if (q + 1 < kBlocks) ask(q + 1);
        if (kHalves == 1 || l16 / kRows == q % kHalves)
#pragma unroll
            for (int f = 0; f < kFrags; ++f)
                *reinterpret_cast<v4f*>(at(l16 % kRows, f * 4 + kg)) = acc[i + f][j];
        const v4f lo = *reinterpret_cast<const v4f*>(at(r, 2 * c)), hi = *reinterpret_cast<const v4f*>(at(r, 2 * c + 1));
        const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        int row, col;
        place(q, row, col);
        if (row < rows && col < cols) put(row, col, v, x[q & 1]);
    }
}

// The same for rows that are no whole vectors.  The loop is rolled (the block is
// picked by a chain of branches), so that `put` stands in the code once.
template <class TL, class Put>
__device__ __forceinline__ void put_blocks(const v4f (&acc)[TL::TN][TL::TM], int wm, int wn, int rows, int cols,
                                           uint8_t* out, Put put) {
    constexpr int TM = TL::TM, TN = TL::TN;
    static_assert(TN % 2 == 0, "column blocks in pairs");
    const int lane = fresh_lane(), l16 = lane & 15, kg = lane >> 4;
    const int r = lane / 4, p = (lane & 3) * 2;
#pragma unroll 1
    for (int q = 0; q < TM * TN / 2; ++q) {
        auto write = [&](const v4f& a, const v4f& b) {
            *reinterpret_cast<v4f*>(out + l16 * 128 + (swz_chunk<128>(l16, kg) << 4)) = a;
            *reinterpret_cast<v4f*>(out + l16 * 128 + (swz_chunk<128>(l16, kg + 4) << 4)) = b;
        };
#pragma unroll
        for (int j = 0; j < TM; ++j)
#pragma unroll
            for (int i = 0; i < TN / 2; ++i)
                if (q == j * (TN / 2) + i) {
                    // (the empty asm keeps the branches apart: merged, they would pick an address,
                    // and the accumulators would live in memory)
                    v4f a = acc[2 * i][j], b = acc[2 * i + 1][j];
                    __asm__ volatile("" : "+v"(a), "+v"(b));
                    write(a, b);
                }
        const v4f lo = *reinterpret_cast<const v4f*>(out + r * 128 + (swz_chunk<128>(r, p) << 4));
        const v4f hi = *reinterpret_cast<const v4f*>(out + r * 128 + (swz_chunk<128>(r, p + 1) << 4));
        const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        const int row = wm * TM * 16 + q / (TN / 2) * 16 + r, col = wn * TN * 16 + q % (TN / 2) * 32 + p * 4;
        if (row < rows && col < cols) put(row, col, v);
    }
}

// ---------------------------------------------------------------------------
// Few tiles, or few rows: a small tile's depth is split over the waves of its workgroup.
// Each wave takes every WAVES-th stage through SLOTS slots of its own, without a barrier,
// and holds the whole tile; the waves' sums are joined in LDS in wave order.
template <int BM_, int BN_, int WAVES_, int SLOTS_, bool AWIDE_, bool BWIDE_>
struct SplitTile {
    static constexpr int BM = BM_, BN = BN_, kWaves = WAVES_, kThreads = kWave * kWaves, kSlots = SLOTS_;
    static constexpr int TM = BM / 16, TN = BN / 16;
    using A = Operand<BM, AWIDE_, 1>;
    using B = Operand<BN, BWIDE_, 1>;
    static constexpr int kStage = A::kBytes + B::kBytes, kLoads = A::kLoads + B::kLoads;
    static constexpr int kPitch = BN + 4;  // floats a row of a wave's sums
    static constexpr int kRing = kWaves * kSlots * kStage, kSums = kWaves * BM * kPitch * 4;
    static constexpr int kLds = kRing > kSums ? kRing : kSums;
};

// One tile: put(row, col, v) is called with 8 neighbouring columns of its sums.
template <class TL, class Job, class Put>
__device__ __forceinline__ void run_split(const Job& job, typename Job::Coord c, uint8_t* s_ring, Put put) {
    constexpr int TM = TL::TM, TN = TL::TN;
    using A = typename TL::A;
    using B = typename TL::B;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t ring0 = (uint32_t)__builtin_amdgcn_readfirstlane(gemm::lds_addr(s_ring) + wave * TL::kSlots * TL::kStage);

    // this wave's stages: `mine` of them; the producer is at depth `at` of segment c
    const int mine = c.stages > wave ? (c.stages - wave + TL::kWaves - 1) / TL::kWaves : 0;
    int at = wave * kStageDepth, issued = 0, slot_in = 0, slot_out = 0;
    const int64_t sa = A::step(job.lda) / kStageDepth, sb = B::step(job.ldb) / kStageDepth;  // bytes a unit of depth
    const uint32_t lda = (uint32_t)job.lda, ldb = (uint32_t)job.ldb;
    A fa;
    B fb;
    auto load = [&]() {  // the next of its stages into the slot of its turn; past the last one nothing, as zeros
        bool more = issued < mine;
        while (more && at >= c.depth) {  // groups of one expert follow each other, each in whole stages
            at -= (c.depth + kStageDepth - 1) / kStageDepth * kStageDepth;
            more = job.segment(c);
        }
        const int left = more ? c.depth - at : 0;
        if (issued == 0 || left < kStageDepth || at < TL::kWaves * kStageDepth) {
            fa.set(0, lane, c.rows_in, left, lda);
            fb.set(0, lane, c.cols_in, left, ldb);
        }
        const uint64_t pa = (uint64_t)gemm::first_lane64((int64_t)c.a + at * sa);
        const uint64_t pb = (uint64_t)gemm::first_lane64((int64_t)c.b + at * sb);
        const int ra = __builtin_amdgcn_readfirstlane(more ? A::range(c.rows_in, left, c.depth, lda) : 0);
        const int rb = __builtin_amdgcn_readfirstlane(more ? B::range(c.cols_in, left, c.depth, ldb) : 0);
        const v4i da = {(int)(uint32_t)pa, (int)(uint32_t)(pa >> 32), ra, 0x00020000};
        const v4i db = {(int)(uint32_t)pb, (int)(uint32_t)(pb >> 32), rb, 0x00020000};
        const uint32_t slot = (uint32_t)__builtin_amdgcn_readfirstlane(ring0 + slot_in * TL::kStage);
        fa.load_all(da, lda, slot);
        fb.load_all(db, ldb, slot + A::kBytes);
        ++issued;
        slot_in = slot_in + 1 < TL::kSlots ? slot_in + 1 : 0;
        at += TL::kWaves * kStageDepth;
    };
    const uint32_t abase = A::lane_base(lane, 0), bbase = B::lane_base(lane, 0);
    v4f acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    float sum[Job::kSums ? TM : 1] = {};
    bool add_up = false;
    if constexpr (Job::kSums) add_up = job.sums(c);
#pragma unroll
    for (int s = 0; s < TL::kSlots; ++s) load();
    for (int s = 0; s < mine; ++s) {
        const uint32_t ca = ring0 + slot_out * TL::kStage + abase, cb = ca - abase + A::kBytes + bbase;
        slot_out = slot_out + 1 < TL::kSlots ? slot_out + 1 : 0;
        gemm::wait_vmem<(TL::kSlots - 1) * TL::kLoads>();
        __asm__ volatile("" ::: "memory");
        v8b tf[2][TM], nf[2][TN];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int i = 0; i < TN; ++i) nf[k][i] = B::frag(cb, i, k);
#pragma unroll
            for (int j = 0; j < TM; ++j) tf[k][j] = A::frag(ca, j, k);
        }
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the slot may be filled again
        __asm__ volatile("" ::: "memory");
        load();
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int j = 0; j < TM; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(nf[k][i], tf[k][j], acc[i][j], 0, 0, 0);
        if constexpr (Job::kSums)
            if (add_up)
#pragma unroll
                for (int j = 0; j < TM; ++j) sum[j] += frag_sum(tf[0][j]) + frag_sum(tf[1][j]);
    }
    gemm::wait_vmem<0>();  // the last loads have landed: the sums may take their place
    __syncthreads();
    float* sums = reinterpret_cast<float*>(s_ring);
    const int l16 = lane & 15, kg = lane >> 4;
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
            *reinterpret_cast<v4f*>(sums + (wave * TL::BM + j * 16 + l16) * TL::kPitch + i * 16 + kg * 4) = acc[i][j];
    if constexpr (Job::kSums)  // a row's partial sums: beside its columns, by lane group
#pragma unroll
        for (int j = 0; j < TM; ++j)
            sums[(wave * TL::BM + j * 16 + l16) * TL::kPitch + TL::BN + kg] = sum[j];
    __syncthreads();
    if constexpr (Job::kSums)
        if (add_up && (int)threadIdx.x < c.rows_in && threadIdx.x < TL::BM) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < TL::kWaves; ++w)
#pragma unroll
                for (int i = 0; i < 4; ++i) v += sums[(w * TL::BM + (int)threadIdx.x) * TL::kPitch + TL::BN + i];
            job.put_sum(c, (int)threadIdx.x, v);
        }
    constexpr int kPieces = TL::BN / 8;
    for (int q = threadIdx.x; q < TL::BM * kPieces; q += TL::kThreads) {
        const int row = q / kPieces, col = q % kPieces * 8;
        if (row >= c.rows_in || col >= c.cols_in) continue;
        float v[8];
#pragma unroll
        for (int w = 0; w < TL::kWaves; ++w) {
            const float* at8 = sums + (w * TL::BM + row) * TL::kPitch + col;
            const v4f lo = *reinterpret_cast<const v4f*>(at8), hi = *reinterpret_cast<const v4f*>(at8 + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = w == 0 ? lo[i] : v[i] + lo[i];
                v[4 + i] = w == 0 ? hi[i] : v[4 + i] + hi[i];
            }
        }
        put(row, col, v);
    }
}

}  // namespace bf16
}  // namespace mxg
