// gemm_bf16_tile.h -- the K pipeline of the BF16 products: operand stages of 64 in
// depth through two LDS slots filled by direct global->LDS loads, read into the matrix
// core's registers one step ahead.  Device code for gfx950.
//
//  * Matrix core: v_mfma_f32_16x16x32_bf16, accumulating.  Operands trade places as in
//    the FP8 products: the operand whose rows become the output's columns is the
//    instruction's A, so a lane's four results are four neighbouring columns of a row.
//  * An operand is either deep (its rows run along the depth: stage rows of 128 bytes,
//    16-byte pieces XOR-swizzled, read 16 bytes a lane) or wide (the depth is its row
//    index: stage rows of R elements, 32-byte pieces XOR-swizzled, read through the
//    transposing LDS load, which gives a lane four depths of its column).
//  * Loads go through buffer descriptors: a lane whose row, column or depth lies past
//    the operand asks for an offset past the descriptor's range, which reads nothing and
//    leaves zeros in LDS.  So rows and tails of any size need no second path, and what
//    lies behind them (another expert's rows, whatever they hold) takes no part.
//  * A stage is two steps of 32 in depth.  While a step is multiplied, the next step's
//    fragments replace its own, one by one.  Two barriers a stage: behind the first
//    (all waves have read the slot) its slot is filled with the stage after the next;
//    behind the second (the next stage has landed) the next stage's fragments are read.
//    A load has about 1.3 stages to land.  The stages run on across tiles: an epilogue
//    has the next tile's first two stages in flight behind it.
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

// A direct-to-LDS load of 16 bytes a lane (lane l to lds + 16 l) through a buffer descriptor;
// both in scalar registers that no vector instruction has just written.
__device__ __forceinline__ void lds_load(const v4i& desc, uint32_t off, uint32_t lds) {
    __asm__ volatile(
        "s_mov_b32 m0, %2\n\ts_nop 0\n\t"
        "buffer_load_dwordx4 %0, %1, 0 offen lds"
        :
        : "v"(off), "s"(desc), "s"(lds)
        : "memory", "m0");
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
    static_assert(R >= 32, "a wide stage row holds two pieces of 32 bytes at least");

    // Wide rows: the 32-byte pieces of a row are XORed with this, so that the eight rows
    // that half a wave reads at one column ({0..3} and {8..11} beside a multiple of 4)
    // lie in distinct banks.  Rows of 128 and 64 bytes already differ by their address.
    static __device__ __forceinline__ int turn(int row) {
        constexpr int kPieces = kRowBytes / 32;
        if constexpr (kPieces >= 8) return (row & 3) | ((row >> 3) & 1) << 2;
        else if constexpr (kPieces == 4) return ((row >> 1) & 1) | ((row >> 3) & 1) << 1;
        else return (row >> 3) & 1;
    }

    uint32_t off[kLoads];

    static __device__ __forceinline__ int stage_row(int wave, int lane, int j) {
        return (wave + NW * j) * kRows + lane / kLanes;
    }
    // which 16-byte piece of the source row this lane fetches
    static __device__ __forceinline__ int piece(int row, int lane) {
        if constexpr (WIDE) return (lane % kLanes) ^ (turn(row) << 1);
        else return swz_chunk<128>(row, lane % 8);
    }
    // Offsets of a stage at whose base `real` rows (columns) and `depth` deep are left; ld: bytes a source row.
    __device__ __forceinline__ void set(int wave, int lane, int real, int64_t depth, uint32_t ld) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int row = stage_row(wave, lane, j), p = piece(row, lane);
            const int across = WIDE ? p * 8 : row, deep = WIDE ? row : p * 8;
            off[j] = across < real && deep < depth ? (uint32_t)row * ld + p * 16 : kNowhere;
        }
    }
    // bytes the base moves a stage
    static __device__ __forceinline__ int64_t step(int64_t ld) { return WIDE ? kStageDepth * ld : 128; }

    // This lane's part of a fragment's address: rows first .. first + 15 of the output side start
    // at multiples of 16.
    static __device__ __forceinline__ uint32_t lane_base(int lane) {
        const int l16 = lane & 15, kg = lane >> 4;
        if constexpr (WIDE) {
            const int row = kg * 8 + l16 / 4;
            return row * kRowBytes + (turn(row) << 5) + (l16 & 3) * 8;
        } else {
            return l16 * 128 + (swz_chunk<128>(l16, kg) << 4);
        }
    }
    // Fragment of rows 16 f .. 16 f + 15, step (0 or 1), from the stage at `slot`.
    static __device__ __forceinline__ v8b frag(const uint8_t* slot, uint32_t base, int f, int step) {
        if constexpr (WIDE) {
            const uint8_t* p = slot + (base ^ (f << 5)) + step * 32 * kRowBytes;
            typedef v4s __attribute__((address_space(3)))* lp;
            typedef uint8_t __attribute__((address_space(3)))* lb;
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)((lb)p));
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)((lb)p + 4 * kRowBytes));
            union {
                v4s s[2];
                v8b b;
            } u;
            u.s[0] = lo;
            u.s[1] = hi;
            return u.b;
        } else {
            return *reinterpret_cast<const v8b*>(slot + (base ^ (step << 6)) + f * (16 * 128));
        }
    }
};

// A tile of BM x BN outputs by WGM x WGN waves; A gives the rows, B the columns.
template <int BM_, int BN_, int WGM_, int WGN_, bool AWIDE_, bool BWIDE_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_;
    static constexpr bool AWIDE = AWIDE_, BWIDE = BWIDE_;
    static constexpr int kWaves = WGM * WGN, kThreads = kWave * kWaves;
    static constexpr int TM = BM / WGM / 16, TN = BN / WGN / 16;  // fragments a wave
    using A = Operand<BM, AWIDE, kWaves>;
    using B = Operand<BN, BWIDE, kWaves>;
    static constexpr int kStage = A::kBytes + B::kBytes;
    static constexpr int kLoads = A::kLoads + B::kLoads;
    static constexpr int kOut = 2048;  // bytes of LDS a wave's epilogue passes its results through
    static constexpr int kLds = 2 * kStage + kWaves * kOut;
    // column blocks of a stage's second step behind which the two barriers stand
    static constexpr int kRead = TN >= 8 ? 1 : 0, kLanded = TN >= 4 ? TN - 3 : TN - 1;
    // A stage's loads are spread over the column blocks from kRead on, about one a block: the loads'
    // path moves 64 bytes a cycle, and waves that issue faster wait.  How many stand before block i:
    static constexpr int loads_before(int i) { return kLoads * (i - kRead) / (TN - kRead); }
};

// The lane number, made anew where it is needed: what derives from it holds no register
// between stages.
__device__ __forceinline__ int fresh_lane() {
    int l;
    __asm__ volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(l));
    return l;
}

// Runs the tiles of `job`.  Job:
//   Coord        int rows_in, cols_in; int64_t stages (of the whole tile), depth (of the present
//                segment); const uint8_t *a, *b (that segment's first stage)
//   bool next(int64_t& W, Coord&)   the first item from W on that there is, or false
//   bool segment(Coord&)            the tile's next stretch of depth, or false
//   lda, ldb                        bytes a row of the operands
//   void finish(c, acc, wave, lane, out)   epilogue of a wave's accumulators
template <class TL, class Job>
__device__ __forceinline__ void run_tiles(Job& job, uint8_t* s_ring, int64_t first, int64_t step) {
    constexpr int TM = TL::TM, TN = TL::TN;
    using A = typename TL::A;
    using B = typename TL::B;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / TL::WGN, wn = wave % TL::WGN;

    typename Job::Coord cc{};
    int64_t cw = first;
    if (!job.next(cw, cc)) return;  // workgroup-uniform

    // ---- the producer: two stages ahead.  Pointers, offsets and `left` (depth from its stage to
    // the segment's end) are those of its next stage; past the last tile every lane asks for
    // nothing, so that its loads need no branch.
    typename Job::Coord pc = cc;
    int64_t pw = cw, left = 0;
    uint64_t pa = 0, pb = 0;
    uint32_t slot = (uint32_t)__builtin_amdgcn_readfirstlane(gemm::lds_addr(s_ring) + wave * 1024);
    const uint32_t slots = 2 * slot + TL::kStage;  // slot + the other slot
    const int64_t sa = gemm::first_lane64(A::step(job.lda)), sb = gemm::first_lane64(B::step(job.ldb));
    A fa;
    B fb;
    auto offsets = [&]() {
        const int lane = fresh_lane();
        fa.set(wave, lane, pc.rows_in, left, (uint32_t)job.lda);
        fb.set(wave, lane, pc.cols_in, left, (uint32_t)job.ldb);
    };
    auto begin = [&]() {  // the first stage of pc's segment
        pa = (uint64_t)gemm::first_lane64((int64_t)pc.a);
        pb = (uint64_t)gemm::first_lane64((int64_t)pc.b);
        left = gemm::first_lane64(pc.depth);
        offsets();
    };
    auto next_tile = [&](bool more) {
        while (more && pc.stages == 0) {
            pw += step;
            more = job.next(pw, pc);
        }
        if (more) return begin();
        pc.rows_in = pc.cols_in = 0;
        left = (int64_t)1 << 62;
        offsets();
    };
    auto load = [&](int l) {
        const v4i da = {(int)(uint32_t)pa, (int)(uint32_t)(pa >> 32), (int)kNowhere, 0x00020000};
        const v4i db = {(int)(uint32_t)pb, (int)(uint32_t)(pb >> 32), (int)kNowhere, 0x00020000};
        if (l < A::kLoads) lds_load(da, fa.off[l < A::kLoads ? l : 0], slot + l * (TL::kWaves * 1024));
        else lds_load(db, fb.off[l < A::kLoads ? 0 : l - A::kLoads], slot + l * (TL::kWaves * 1024));
    };
    auto load_all = [&]() {
#pragma unroll
        for (int l = 0; l < TL::kLoads; ++l) load(l);
    };
    auto advance = [&]() {  // behind a stage's loads
        slot = slots - slot;
        pa += sa;
        pb += sb;
        left -= kStageDepth;
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
    load_all();
    advance();
    load_all();
    advance();
    stage_barrier<TL::kLoads>();

    // ---- the consumer
    v8b tf[2][TM], nf[TN];
    uint32_t abase, bbase;
    {
        const int lane = threadIdx.x & (kWave - 1);
        abase = A::lane_base(lane);
        bbase = B::lane_base(lane);
    }
    const int a0 = wm * TM, b0 = wn * TN;  // the wave's first fragments
    int cslot = 0;
    auto first_frags = [&](const uint8_t* at) {
#pragma unroll
        for (int i = 0; i < TN; ++i) nf[i] = B::frag(at + A::kBytes, bbase, b0 + i, 0);
#pragma unroll
        for (int j = 0; j < TM; ++j) tf[0][j] = A::frag(at, abase, a0 + j, 0);
    };
    first_frags(s_ring);
    bool drain = false;  // an epilogue's stores are outstanding: counted waits do not hold
    for (;;) {
        const bool live = a0 * 16 < cc.rows_in && b0 * 16 < cc.cols_in;  // wave-uniform
        v4f acc[TN][TM];
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
        const int64_t stages = cc.stages;
        auto read_barrier = [&]() {
            if (drain) gemm::wait_vmem<0>();
            drain = false;
            __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's fragments are in registers
            __asm__ volatile("" ::: "memory");
            __builtin_amdgcn_s_barrier();
            __asm__ volatile("" ::: "memory");
        };
        if (live) {
            for (int64_t kt = 0; kt < stages; ++kt) {
                const uint8_t *cur = s_ring + cslot * TL::kStage, *nxt = s_ring + (cslot ^ 1) * TL::kStage;
#pragma unroll
                for (int i = 0; i < TN; ++i) {
#pragma unroll
                    for (int j = 0; j < TM; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(nf[i], tf[0][j], acc[i][j], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    nf[i] = B::frag(cur + A::kBytes, bbase, b0 + i, 1);
#pragma unroll
                    for (int j = i * TM / TN; j < (i + 1) * TM / TN; ++j) tf[1][j] = A::frag(cur, abase, a0 + j, 1);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int i = 0; i < TN; ++i) {
#pragma unroll
                    for (int j = 0; j < TM; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(nf[i], tf[1][j], acc[i][j], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    if (i == TL::kRead) read_barrier();
                    if (i >= TL::kRead)
#pragma unroll
                        for (int q = TL::loads_before(i); q < TL::loads_before(i + 1); ++q) load(q);
                    if (i == TL::kLanded) {
                        stage_barrier<TL::loads_before(TL::kLanded + 1)>();
                        nf[0] = B::frag(nxt + A::kBytes, bbase, b0, 0);
#pragma unroll
                        for (int j = 0; j < TM; ++j) tf[0][j] = A::frag(nxt, abase, a0 + j, 0);
#pragma unroll
                        for (int f = 1; f <= i; ++f) nf[f] = B::frag(nxt + A::kBytes, bbase, b0 + f, 0);
                    }
                    if (i > TL::kLanded) nf[i] = B::frag(nxt + A::kBytes, bbase, b0 + i, 0);
                    __builtin_amdgcn_sched_barrier(0);
                }
                advance();
                cslot ^= 1;
            }
            job.template finish<TL>(cc, acc, wm, wn, s_ring + 2 * TL::kStage + wave * TL::kOut);
        } else if (stages > 0) {
            for (int64_t kt = 0; kt < stages; ++kt) {
                read_barrier();
                load_all();
                stage_barrier<TL::kLoads>();
                advance();
                cslot ^= 1;
            }
            first_frags(s_ring + cslot * TL::kStage);  // the next tile's
        }
        drain = true;
        cw += step;
        if (!job.next(cw, cc)) break;
    }
    gemm::wait_vmem<0>();  // no load may land once the workgroup's LDS belongs to another
}

// A wave's accumulators through its LDS buffer, 16 rows x 32 columns at a time: calls
// put(row, col, v) with 8 neighbouring columns of a row of the tile.  The loop is rolled
// (the block is picked by a switch), so that `put` stands in the code once.
template <class TL, class Put>
__device__ __forceinline__ void put_blocks(const v4f (&acc)[TL::TN][TL::TM], int wm, int wn, uint8_t* out, Put put) {
    constexpr int TM = TL::TM, TN = TL::TN;
    static_assert(TN % 2 == 0, "column blocks in pairs");
    const int lane = fresh_lane(), l16 = lane & 15, kg = lane >> 4;
    const int r = lane / 4, p = (lane & 3) * 2;
#pragma unroll 1
    for (int q = 0; q < TM * TN / 2; ++q) {
        auto write = [&](const v4f& x, const v4f& y) {
            *reinterpret_cast<v4f*>(out + l16 * 128 + (swz_chunk<128>(l16, kg) << 4)) = x;
            *reinterpret_cast<v4f*>(out + l16 * 128 + (swz_chunk<128>(l16, kg + 4) << 4)) = y;
        };
#pragma unroll
        for (int j = 0; j < TM; ++j)
#pragma unroll
            for (int i = 0; i < TN / 2; ++i)
                if (q == j * (TN / 2) + i) {
                    // (the empty asm keeps the branches apart: merged, they would pick an address,
                    // and the accumulators would live in memory)
                    v4f x = acc[2 * i][j], y = acc[2 * i + 1][j];
                    __asm__ volatile("" : "+v"(x), "+v"(y));
                    write(x, y);
                }
        const v4f lo = *reinterpret_cast<const v4f*>(out + r * 128 + (swz_chunk<128>(r, p) << 4));
        const v4f hi = *reinterpret_cast<const v4f*>(out + r * 128 + (swz_chunk<128>(r, p + 1) << 4));
        const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        put(wm * TM * 16 + q / (TN / 2) * 16 + r, wn * TN * 16 + q % (TN / 2) * 32 + p * 4, v);
    }
}

}  // namespace bf16
}  // namespace mxg
