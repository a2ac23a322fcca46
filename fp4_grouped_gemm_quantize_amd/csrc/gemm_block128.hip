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
//    cores' issue time and run beside them.
//  * Operands trade places: the weights are the instruction's A, the tokens its
//    B, so a lane's four results are four columns of one token.  A lane then
//    needs one scale per 16-token block (the token's times the wave's weight
//    scale, which is uniform), and its results pack to 8 bytes of BF16.
//  * Tiles, the direct global->LDS ring, the ragged tile map, the XCD-aware
//    order and the persistent schedule are those of the rowwise GEMM
//    (gemm_common.h); a ring stage is 128 K bytes per row, one scale block.
//  * A's scales: eight blocks of the tile's rows at a time through registers
//    into LDS, rows innermost, so that a lane's read is conflict-free.
#include "gemm_common.h"

namespace mxg {

using namespace gemm;

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
constexpr int kSB = 128;          // stage bytes per row: one scale block
constexpr int kSclBlocks = 8;     // scale blocks per LDS chunk

// BM tokens x BN columns, WGM x WGN waves.
template <int BM_, int BN_, int WGM_, int WGN_>
struct BTile {
    static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_;
    static constexpr int kWaves = WGM * WGN, kThreads = kWave * kWaves;
    static constexpr int WTM = BM / WGM, WTN = BN / WGN;
    static constexpr int TM = WTM / 16, TN = WTN / 16;
    static_assert(128 % WTN == 0, "a wave's columns lie in one weight scale block");
    static_assert(BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0, "loader: whole row groups per wave");
    static_assert(kWaves % 2 == 0, "per-lane chunk independent of the load index");
};

// One 16-row fragment of a 128-deep block: lane l holds row l % 16, chunks l / 16
// and l / 16 + 4 (both operands alike, so the order of K inside the block is free).
__device__ __forceinline__ v8i load_frag16(const uint8_t* __restrict__ base, int row, int kg) {
    const int at = swz<kSB>(row, kg);
    const uint4 x0 = *reinterpret_cast<const uint4*>(base + at);
    const uint4 x1 = *reinterpret_cast<const uint4*>(base + (at ^ 64));
    return v8i{(int)x0.x, (int)x0.y, (int)x0.z, (int)x0.w, (int)x1.x, (int)x1.y, (int)x1.z, (int)x1.w};
}

__device__ __forceinline__ v4f mma128(const v8i& n, const v8i& t) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(n, t, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// KTAIL: K is not a multiple of 128; the last stage goes through registers with
// its tail zeroed.
template <class TL, bool KTAIL>
__global__ __launch_bounds__(TL::kThreads, 1) void block128_kernel(const GemmArgs args) {
    constexpr int BM = TL::BM, BN = TL::BN, NW = TL::kWaves, NT = TL::kThreads;
    constexpr int WTM = TL::WTM, WTN = TL::WTN, TM = TL::TM, TN = TL::TN;
    constexpr int kAStage = BM * kSB, kBStage = BN * kSB, kStage = kAStage + kBStage;
    constexpr int A_J = BM / 8 / NW, B_J = BN / 8 / NW;
    constexpr int kSclPer = BM * kSclBlocks / NT;  // scales a thread loads per chunk
    static_assert(BM * kSclBlocks % NT == 0 && kSclBlocks % kSclPer == 0, "scale chunk: whole pieces per thread");
    __shared__ __attribute__((aligned(16))) uint8_t s_ring0[kStage];
    __shared__ __attribute__((aligned(16))) uint8_t s_ring1[kStage];
    __shared__ float s_scl[2][kSclBlocks][BM];
    __shared__ uint32_t s_pre[kMaxGroups + 1];
    __shared__ uint32_t s_wave[NW];

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / TL::WGN, wn = wave % TL::WGN;
    const int l16 = lane & 15, kg = lane >> 4;

    build_tile_prefix<NT, BM>(args, s_pre, s_wave);
    const int64_t total_tiles = (int64_t)s_pre[args.G] * args.ntiles_n;
    const int64_t K = args.K;
    const int nkt = (int)((K + kSB - 1) / kSB);
    const int64_t nnb = (args.N + 127) / 128;

    const WorkSplit ws = work_split(total_tiles, gridDim.x);
    for (int64_t W = xcd_remap(blockIdx.x, gridDim.x); W < ws.items; W += gridDim.x) {
        const TileCoord tc = uniform_coord(locate_item<BM, BN>(args, s_pre, ws, W));
        if (tc.cols_in <= 0) continue;  // the empty second half of a last, narrow tile (uniform)
        const int64_t m0 = tc.m0, n0 = tc.n0;
        const int rows_in = tc.rows_in, cols_in = tc.cols_in;
        const bool wave_live = wm * WTM < rows_in && wn * WTN < cols_in;  // wave-uniform

        // operand sources: uniform base + 32-bit lane offsets; rows past the
        // group and columns past N re-read the last real one
        const uint8_t* a_base = args.a + m0 * K;
        const uint8_t* b_base = args.b + ((int64_t)tc.e * args.N + n0) * K;
        const int r0 = wave * 8 + lane / 8;
        const int chunk = swz_chunk<kSB>(r0, lane % 8);
        uint32_t a_off[A_J], b_off[B_J];
#pragma unroll
        for (int j = 0; j < A_J; ++j) {
            const int r = r0 + 8 * NW * j;
            a_off[j] = (uint32_t)(r < rows_in ? r : rows_in - 1) * (uint32_t)K + chunk * 16;
        }
#pragma unroll
        for (int j = 0; j < B_J; ++j) {
            const int r = r0 + 8 * NW * j;
            b_off[j] = (uint32_t)(r < cols_in ? r : cols_in - 1) * (uint32_t)K + chunk * 16;
        }
        auto issue_stage = [&](int kt, uint8_t* slot) {
            const uint8_t* ak = a_base + (int64_t)kt * kSB;
            const uint8_t* bk = b_base + (int64_t)kt * kSB;
#pragma unroll
            for (int j = 0; j < A_J; ++j)
                __builtin_amdgcn_global_load_lds((gptr_t)(ak + a_off[j]), (lptr_t)(slot + (wave + NW * j) * 1024), 16,
                                                 0, 0);
#pragma unroll
            for (int j = 0; j < B_J; ++j)
                __builtin_amdgcn_global_load_lds((gptr_t)(bk + b_off[j]),
                                                 (lptr_t)(slot + kAStage + (wave + NW * j) * 1024), 16, 0, 0);
        };
        auto put_tail = [&](int kt, uint8_t* slot) {
            const bool in = (int64_t)kt * kSB + chunk * 16 < K;
            uint4 ta[A_J], tb[B_J];
#pragma unroll
            for (int j = 0; j < A_J; ++j)
                ta[j] = in ? *reinterpret_cast<const uint4*>(a_base + (int64_t)kt * kSB + a_off[j])
                           : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < B_J; ++j)
                tb[j] = in ? *reinterpret_cast<const uint4*>(b_base + (int64_t)kt * kSB + b_off[j])
                           : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < A_J; ++j) *reinterpret_cast<uint4*>(slot + (wave + NW * j) * 1024 + lane * 16) = ta[j];
#pragma unroll
            for (int j = 0; j < B_J; ++j)
                *reinterpret_cast<uint4*>(slot + kAStage + (wave + NW * j) * 1024 + lane * 16) = tb[j];
        };
        auto put_stage = [&](int kt, uint8_t* slot) {
            if (KTAIL && kt == nkt - 1) put_tail(kt, slot);
            else issue_stage(kt, slot);
        };

        // A's scales: thread tid loads kSclPer consecutive blocks of one row
        const int srow = tid * kSclPer / kSclBlocks, sblk = tid * kSclPer % kSclBlocks;
        const float* s_src = static_cast<const float*>(args.as) +
                             (m0 + (srow < rows_in ? srow : rows_in - 1)) * (int64_t)nkt + sblk;
        float sreg[kSclPer];
        auto load_scales = [&](int c) {
#pragma unroll
            for (int i = 0; i < kSclPer; ++i)
                sreg[i] = c * kSclBlocks + sblk + i < nkt ? s_src[c * kSclBlocks + i] : 0.0f;
        };
        auto store_scales = [&](int c) {
#pragma unroll
            for (int i = 0; i < kSclPer; ++i) s_scl[c & 1][sblk + i][srow] = sreg[i];
        };
        // the wave's weight scales, one per stage (wave-uniform)
        const float* b_scl = static_cast<const float*>(args.bs) +
                             ((int64_t)tc.e * nnb + (wave_live ? (n0 + wn * WTN) / 128 : n0 / 128)) * nkt;

        v4f acc[TN][TM];
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

        put_stage(0, s_ring0);
        load_scales(0);
        store_scales(0);
        wait_vmem<0>();
        __syncthreads();

        auto stage = [&](int kt, const uint8_t* cur, uint8_t* nxt) {
            if (kt + 1 < nkt) put_stage(kt + 1, nxt);
            const bool more = kt % kSclBlocks == kSclBlocks - 2 && kt + 2 < nkt;
            if (more) load_scales(kt / kSclBlocks + 1);
            if (wave_live) {
                const float sb = b_scl[kt];
                float s[TM];
                v8i tf[TM];
#pragma unroll
                for (int j = 0; j < TM; ++j) {
                    s[j] = s_scl[(kt / kSclBlocks) & 1][kt % kSclBlocks][wm * WTM + j * 16 + l16] * sb;
                    tf[j] = load_frag16(cur, wm * WTM + j * 16 + l16, kg);
                }
                v4f part[2][TM];
#pragma unroll
                for (int i = 0; i <= TN; ++i) {
                    if (i < TN) {
                        const v8i nf = load_frag16(cur + kAStage, wn * WTN + i * 16 + l16, kg);
#pragma unroll
                        for (int j = 0; j < TM; ++j) part[i & 1][j] = mma128(nf, tf[j]);
                    }
                    if (i > 0) {
#pragma unroll
                        for (int j = 0; j < TM; ++j)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                acc[i - 1][j][r] = fmaf(part[(i - 1) & 1][j][r], s[j], acc[i - 1][j][r]);
                    }
                }
            }
            if (more) store_scales(kt / kSclBlocks + 1);
            stage_barrier<0>();
        };
        for (int kt = 0; kt < nkt; kt += 2) {
            stage(kt, s_ring0, s_ring1);
            if (kt + 1 < nkt) stage(kt + 1, s_ring1, s_ring0);
        }

        // ---- epilogue: BF16 rows staged in the ring (free after the last
        // barrier), 16-byte pieces XOR-swizzled by the row so that the lanes'
        // 8-byte writes (16 rows at one column) and the readers' whole rows are
        // both conflict-free, then written out in 16-byte pieces
        if ((args.N & 7) == 0) {
            constexpr int kPieces = BN / 8;
            constexpr int kRowsPerSlot = kStage / (BN * 2);
            static_assert(2 * kRowsPerSlot >= BM, "the tile's rows fit the ring");
            auto piece = [&](int row, int p) -> uint8_t* {
                uint8_t* base = row < kRowsPerSlot ? s_ring0 : s_ring1;
                return base + (row % kRowsPerSlot) * (BN * 2) + ((p ^ (row & 15)) << 4);
            };
            if (wave_live) {
#pragma unroll
                for (int j = 0; j < TM; ++j) {
                    const int row = wm * WTM + j * 16 + l16;
#pragma unroll
                    for (int i = 0; i < TN; ++i) {
                        const int col = wn * WTN + i * 16 + kg * 4;
                        *reinterpret_cast<uint2*>(piece(row, col / 8) + (col & 4) * 2) =
                            make_uint2(f32x2_to_bf16x2(acc[i][j][0], acc[i][j][1]),
                                       f32x2_to_bf16x2(acc[i][j][2], acc[i][j][3]));
                    }
                }
            }
            __syncthreads();
#pragma unroll 1
            for (int q = tid; q < BM * kPieces; q += NT) {
                const int row = q / kPieces, p = q % kPieces;
                if (row < rows_in && p * 8 < cols_in)
                    store_stream16(args.c + (m0 + row) * args.N + n0 + p * 8,
                                   *reinterpret_cast<const uint4*>(piece(row, p)));
            }
            __syncthreads();  // the ring is reused by the next tile
        } else if (wave_live) {
            // rows of c that do not start on 16 bytes: element stores
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int row = wm * WTM + j * 16 + l16;
                if (row >= rows_in) continue;
#pragma unroll
                for (int i = 0; i < TN; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int col = wn * WTN + i * 16 + kg * 4 + r;
                        if (col < cols_in)
                            args.c[(m0 + row) * args.N + n0 + col] = (uint16_t)f32_to_bf16(acc[i][j][r]);
                    }
            }
        }
    }
}

template <class TL>
hipError_t launch_tile(const GemmProblem& p, hipStream_t stream, int mband, int per_cu) {
    auto kernel = p.K % kSB ? block128_kernel<TL, true> : block128_kernel<TL, false>;
    int64_t grid = 0;
    const GemmArgs a = make_args(p, TL::BM, TL::BN, mband, per_cu, &grid);
    if (grid <= 0) return hipSuccess;
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(TL::kThreads), 0, stream, a);
    return hipGetLastError();
}

using TileLarge = BTile<256, 256, 4, 2>;
using TileSmall = BTile<64, 128, 1, 4>;

}  // namespace

hipError_t launch_grouped_gemm_block128(const GemmProblem& p, hipStream_t stream) {
    const int64_t groups = p.G < p.T ? p.G : p.T;
    const int64_t avg = groups > 0 ? p.T / groups : p.T;
    const int64_t rows = p.max_rows_hint > avg ? (avg + p.max_rows_hint) / 2 : avg;
    if (rows >= 128) return launch_tile<TileLarge>(p, stream, 4, 1);
    return launch_tile<TileSmall>(p, stream, 1 << 30, 2);
}

}  // namespace mxg
