// route.hip -- the router (top-k expert choice and its gradient) and the routing
// plan (a stable counting sort of the slots by expert), for gfx950.
//
// (Struct_ep_dispatch_mxfp4: topk_ids, row_offsets and src_info; the pages name
//  these arrays and do not say how they are made.)
//
// All three are small integer or scalar jobs over [tokens, experts] or [slots]
// arrays, bound by latency: each is one launch (the sort of very many slots four),
// without workspace, and results do not depend on timing.  Measured (a kernel's time
// on the device, in a trace): choice of 8 from 128 experts for 8192 tokens 5.1 us and
// its gradient 4.8, choice of 8 from 64 under a bias for 64 tokens 4.6.  For 65536
// tokens 18 and 14 (38 MB and 71): there the choice's rounds bound it, which walk a
// lane's elements three times each (maximum, index, clearing).
#include <type_traits>

#include "mxg_device.h"
#include "mxg_internal.h"

namespace mxg {

namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// Cross-lane exchange inside a token's LPT lanes.  Within 16 lanes (a DPP row)
// the four steps are register moves: lane ^ 1 and lane ^ 2 (quad permutes),
// then the mirrors within 8 and 16 lanes, which pair values that are by then
// equal inside each quad / half.  Wider groups add shuffles over 16 and 32.
template <int STEP>
__device__ __forceinline__ uint32_t exchange(uint32_t v) {
    if constexpr (STEP == 0) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true);
    else if constexpr (STEP == 1) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true);
    else if constexpr (STEP == 2) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true);
    else if constexpr (STEP == 3) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true);
    else return (uint32_t)__shfl_xor((int)v, 1 << STEP, kWave);
}
template <int STEP>
__device__ __forceinline__ uint64_t exchange(uint64_t v) {
    return ((uint64_t)exchange<STEP>((uint32_t)(v >> 32)) << 32) | exchange<STEP>((uint32_t)v);
}
template <int STEP>
__device__ __forceinline__ float exchange(float v) {
    return __uint_as_float(exchange<STEP>(__float_as_uint(v)));
}
template <int STEP>
__device__ __forceinline__ double exchange(double v) {
    return __longlong_as_double((long long)exchange<STEP>((uint64_t)__double_as_longlong(v)));
}

// v combined over a token's LPT lanes by f (the result in every lane).
template <int LPT, class T, class F>
__device__ __forceinline__ T reduce(T v, F f) {
    v = f(v, exchange<0>(v));
    v = f(v, exchange<1>(v));
    v = f(v, exchange<2>(v));
    v = f(v, exchange<3>(v));
    if constexpr (LPT == 64) {
        v = f(v, exchange<4>(v));
        v = f(v, exchange<5>(v));
    }
    return v;
}
template <int LPT, class T>
__device__ __forceinline__ T sum_over(T v) {
    return reduce<LPT>(v, [](T a, T b) { return a + b; });
}
template <int LPT>
__device__ __forceinline__ float max_over(float v) {
    return reduce<LPT>(v, [](float a, float b) { return fmaxf(a, b); });
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) { *p = (uint16_t)f32_to_bf16(v); }

// Keys in an order that unsigned comparison keeps, 0 for a value that may not
// be chosen (-infinity, NaN): every other value maps above 0.  Adding zero
// turns -0 into +0, which compare equal.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return v > -INFINITY ? ((u >> 31) ? ~u : u | 0x80000000u) : 0u;
}
// Biased scores are compared as they are, -infinity for what may not be chosen.
__device__ __forceinline__ double order_key(double v) { return v > -(double)INFINITY ? v : -(double)INFINITY; }
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }
// log(1 / (1 + e^-x)), exact where the sigmoid itself underflows
__device__ __forceinline__ float log_sigmoid(float x) { return fminf(x, 0.0f) - log1pf(expf(-fabsf(x))); }

// ---------------------------------------------------------------------------
// LPT lanes hold a token's logits, expert i in lane i % LPT (element i / LPT),
// so loads are coalesced and a lane's elements rise with their index.  Each of
// the top_k rounds takes the largest key over the lane's own elements and the
// token's lanes, then the lowest index that has it, and clears that one: maxima
// and minima alone, which the exchanges' register moves fold into (carrying each
// key's index through the maximum: 65536 x 128, 8 of them, 20.8 us instead of
// 16.1; 8192 x 128, 32 of them, 35 instead of 21).  16 lanes a token hold four
// tokens a wave, so a round serves four.  Lane j ends with slot j, so 16 lanes
// serve top_k <= 16.
template <class LT, int LPT, int VPL, bool BIASED>
__global__ __launch_bounds__(kThreads) void topk_kernel(const LT* __restrict__ logits, const float* __restrict__ bias,
                                                        int64_t ntok, int E, int top_k, int score, bool renorm,
                                                        float scale, int32_t* __restrict__ ids,
                                                        float* __restrict__ weights) {
    const int sub = threadIdx.x % LPT;
    for (int64_t t0 = (int64_t)blockIdx.x * (kThreads / LPT); t0 < ntok; t0 += (int64_t)gridDim.x * (kThreads / LPT)) {
        const int64_t t = t0 + threadIdx.x / LPT;
        using Key = typename std::conditional<BIASED, double, uint32_t>::type;
        const Key none = BIASED ? (Key)-INFINITY : (Key)0;
        const bool on = t < ntok;  // the lanes of a token past the end stay for the exchanges
        const LT* row = logits + (on ? t : 0) * E;

        float x[VPL];
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int i = v * LPT + sub;
            x[v] = on && i < E ? load_logit(row + i) : -INFINITY;
        }
        float b[BIASED ? VPL : 1];  // loaded beside the logits, not behind the scores (64 tokens: 0.5 us less)
        if constexpr (BIASED) {
#pragma unroll
            for (int v = 0; v < VPL; ++v) b[v] = bias[v * LPT + sub < E ? v * LPT + sub : 0];
        }
        float top = x[0];
#pragma unroll
        for (int v = 1; v < VPL; ++v) top = fmaxf(top, x[v]);
        top = max_over<LPT>(top);

        Key key[VPL];
        if constexpr (BIASED) {
            double total = 1.0;
            if (score == 0) {
                double z = 0.0;
#pragma unroll
                for (int v = 0; v < VPL; ++v)
                    if (v * LPT + sub < E) z += exp((double)x[v] - (double)top);
                total = sum_over<LPT>(z);
            }
#pragma unroll
            for (int v = 0; v < VPL; ++v) {
                const int i = v * LPT + sub;
                key[v] = none;
                if (i < E && x[v] > -INFINITY) {
                    const double s = score == 0 ? exp((double)x[v] - (double)top) / total
                                                : 1.0 / (1.0 + exp(-(double)x[v]));
                    key[v] = order_key(s + (double)b[v]);
                }
            }
        } else {
#pragma unroll
            for (int v = 0; v < VPL; ++v) key[v] = order_key(x[v]);
        }

        int32_t my_id = -1;
        for (int k = 0; k < top_k; ++k) {
            Key best = key[0];
#pragma unroll
            for (int v = 1; v < VPL; ++v) best = larger(best, key[v]);
            best = reduce<LPT>(best, [](Key p, Key q) { return larger(p, q); });
            uint32_t at = ~0u;
#pragma unroll
            for (int v = VPL - 1; v >= 0; --v) at = key[v] == best ? (uint32_t)(v * LPT + sub) : at;
            at = reduce<LPT>(at, [](uint32_t p, uint32_t q) { return p < q ? p : q; });
            if (sub == k) my_id = best > none ? (int32_t)at : -1;
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                if ((uint32_t)(v * LPT + sub) == at) key[v] = none;
        }

        const bool live = my_id >= 0;
        const float mine = live ? load_logit(row + my_id) : 0.0f;
        float w;
        if (renorm) {
            const float l = !live ? -INFINITY : score == 0 ? mine : log_sigmoid(mine);
            const float m = max_over<LPT>(l);
            w = live ? expf(l - m) : 0.0f;
            w = w / sum_over<LPT>(w);
        } else if (score == 0) {
            float z = 0.0f;
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                if (v * LPT + sub < E) z += expf(x[v] - top);
            w = expf(mine - top) / sum_over<LPT>(z);
        } else {
            w = sigmoid(mine);
        }
        if (on && sub < top_k) {
            ids[t * top_k + sub] = my_id;
            weights[t * top_k + sub] = live ? scale * w : 0.0f;
        }
    }
}

// The gradient: lane j forms slot j's g_j (the gradient of the log of its
// score, and for the sigmoid of its logit), then every lane adds the slots that
// name one of its own experts.  The logits are read whole only where the
// gradient needs them (softmax without renormalisation).
template <class LT, int LPT, int VPL>
__global__ __launch_bounds__(kThreads) void topk_backward_kernel(const LT* __restrict__ logits,
                                                                 const int32_t* __restrict__ ids,
                                                                 const float* __restrict__ dweights, int64_t ntok,
                                                                 int E, int top_k, int score, bool renorm, float scale,
                                                                 LT* __restrict__ dlogits) {
    const int sub = threadIdx.x % LPT;
    for (int64_t t0 = (int64_t)blockIdx.x * (kThreads / LPT); t0 < ntok; t0 += (int64_t)gridDim.x * (kThreads / LPT)) {
        const int64_t t = t0 + threadIdx.x / LPT;
        const bool on = t < ntok;
        const LT* row = logits + (on ? t : 0) * E;
        int32_t id = -1;
        float d = 0.0f, mine = -INFINITY;
        if (on && sub < top_k) {
            id = ids[t * top_k + sub];
            if (id < 0 || id >= E) id = -1;
            if (id >= 0) {
                mine = load_logit(row + id);
                d = scale * dweights[t * top_k + sub];
            }
        }
        if (mine == -INFINITY) id = -1;  // a score of 0: its weight is 0 and stays so
        const bool live = id >= 0;

        float g = 0.0f, top = 0.0f, total = 1.0f, x[VPL];
        const bool whole = score == 0 && !renorm;
        if (whole) {
#pragma unroll
            for (int v = 0; v < VPL; ++v) {
                const int i = v * LPT + sub;
                x[v] = on && i < E ? load_logit(row + i) : -INFINITY;
            }
            top = x[0];
#pragma unroll
            for (int v = 1; v < VPL; ++v) top = fmaxf(top, x[v]);
            top = max_over<LPT>(top);
            float z = 0.0f;
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                if (v * LPT + sub < E) z += expf(x[v] - top);
            total = sum_over<LPT>(z);
            g = live ? expf(mine - top) / total * d : 0.0f;
        } else if (renorm) {
            const float l = !live ? -INFINITY : score == 0 ? mine : log_sigmoid(mine);
            const float m = max_over<LPT>(l);
            float r = live ? expf(l - m) : 0.0f;
            r = r / sum_over<LPT>(r);
            const float inner = sum_over<LPT>(live ? r * d : 0.0f);
            g = live ? r * (d - inner) : 0.0f;
        } else {
            g = live ? sigmoid(mine) * d : 0.0f;
        }
        if (score == 1 && live) g *= sigmoid(-mine);
        const float all = whole ? sum_over<LPT>(g) : 0.0f;

        float acc[VPL];
#pragma unroll
        for (int v = 0; v < VPL; ++v) acc[v] = 0.0f;
        const int first = (threadIdx.x & (kWave - 1)) - sub;  // the token's first lane in the wave
        for (int k = 0; k < top_k; ++k) {
            const int32_t ik = __shfl(id, first + k, kWave);
            const float gk = __shfl(g, first + k, kWave);
#pragma unroll
            for (int v = 0; v < VPL; ++v) acc[v] += ik == v * LPT + sub ? gk : 0.0f;
        }
        if (!on) continue;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int i = v * LPT + sub;
            if (i >= E) continue;
            float out = acc[v];
            if (whole && all != 0.0f) out -= expf(x[v] - top) / total * all;
            store_logit(dlogits + t * E + i, out);
        }
    }
}

// ---------------------------------------------------------------------------
// Stable counting sort of n slots by expert id, one workgroup per expert (very many
// slots: see sort_count_kernel).
// Workgroup e reads every id (the whole list is a few hundred KB at most and
// stays in L2): the ids below e give its first row, the ids equal to e, in slot
// order, its rows.  A wave owns a contiguous stretch of the slots and takes 512
// of them a step, eight a lane, so the rank of a slot is the matches of the waves
// before, of its wave's steps before, of the lanes before (a scan of the lanes'
// counts) and of its own lane's ids before.  Reading the list once per expert
// needs neither a workspace nor a second launch, nor atomics whose speed falls
// when one expert takes most slots.  Bound by instruction issue (a compare for
// each of the two questions, the counts on the scalar unit).  The matches are kept
// as eight bits a step, of 8 steps a wave at most (65536 slots; longer lists go to
// the kernels below).  Measured, 65536 slots of 128 experts: 8.2 us (21
// with one id a lane and step, 13 with four and a ballot for each, 26 with the
// slots of an expert split over workgroups); 1024 slots of 64: 3.2 us.
constexpr int kKeep = 8, kIds = 8;

// Eight consecutive ids, -1 past the end.  inside (wave-uniform): all are before
// it.  No branch either way, so a wave's loads leave together.
typedef int ids4 __attribute__((ext_vector_type(4), aligned(4)));
struct Ids {
    int32_t v[kIds];
};
__device__ __forceinline__ Ids load_ids(const int32_t* __restrict__ ids, int64_t i, int64_t n, bool inside) {
    Ids r;
    if (inside) {
        const ids4 lo = *reinterpret_cast<const ids4*>(ids + i), hi = *reinterpret_cast<const ids4*>(ids + i + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r.v[j] = lo[j];
            r.v[j + 4] = hi[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < kIds; ++j) {
            const int32_t x = ids[i + j < n ? i + j : n - 1];
            r.v[j] = i + j < n ? x : -1;
        }
    }
    return r;
}

// The matches of eight ids with e, a bit each; counts the ids below e over the
// wave (a negative id is a large one).
__device__ __forceinline__ uint32_t match(const Ids& id, uint32_t e, uint32_t& less) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kIds; ++j) {
        less += (uint32_t)__popcll(__ballot((uint32_t)id.v[j] < e));
        m |= (uint32_t)id.v[j] == e ? 1u << j : 0u;
    }
    return m;
}

// Sum over the lanes up to and with this one: shifts inside rows of 16, then the
// rows' last lanes broadcast on.
__device__ __forceinline__ uint32_t lane_scan(uint32_t v) {
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false);  // row_shr:1
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false);  // row_bcast:15 into rows 1, 3
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false);  // row_bcast:31 into rows 2, 3
    return v;
}

template <int NT>
__global__ __launch_bounds__(NT) void sort_kernel(const int32_t* __restrict__ ids, int64_t n, int E,
                                                  uint32_t* __restrict__ off, int32_t* __restrict__ row_of_slot,
                                                  int32_t* __restrict__ slot_of_row) {
    constexpr int NW = NT / kWave;
    __shared__ uint32_t s_less[NW], s_same[NW];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t e = blockIdx.x;
    constexpr int kStep = kIds * kWave;
    const int steps = (int)((n + NW * kStep - 1) / (NW * kStep));  // per wave, at most kKeep
    const int64_t base = (int64_t)wave * steps * kStep + lane * kIds;  // this lane's first slot
    const bool inside = (int64_t)(wave + 1) * steps * kStep <= n;

    uint32_t less = 0, same = 0, hits[kKeep / 4] = {};  // hits: eight bits a step
    Ids v[kKeep];
    if (inside) {
#pragma unroll
        for (int s = 0; s < kKeep; ++s)
            if (s < steps) v[s] = load_ids(ids, base + (int64_t)s * kStep, n, true);
    } else {
#pragma unroll
        for (int s = 0; s < kKeep; ++s)
            if (s < steps) v[s] = load_ids(ids, base + (int64_t)s * kStep, n, false);
    }
#pragma unroll
    for (int s = 0; s < kKeep; ++s)
        if (s < steps) hits[s / 4] |= match(v[s], e, less) << (8 * (s % 4));
#pragma unroll
    for (int h = 0; h < kKeep / 4; ++h) same += __popc(hits[h]);
    same = (uint32_t)__builtin_amdgcn_readlane((int)lane_scan(same), kWave - 1);
    if (lane == 0) {
        s_less[wave] = less;
        s_same[wave] = same;
    }
    __syncthreads();
    uint32_t first = 0, run = 0, all_same = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        first += s_less[w];
        run += w < wave ? s_same[w] : 0;
        all_same += s_same[w];
    }
    const uint32_t total = first + all_same;  // of the last expert: the slots that were not dropped
    if (threadIdx.x == 0) {
        off[e] = first;
        if ((int)e == E - 1) off[E] = total;
    }
    run += first;
    auto place = [&](int64_t i, uint32_t m) {  // the matches m of the step whose ids start at slot i
        if (!__any(m != 0)) return;
        const uint32_t mine = __popc(m), upto = lane_scan(mine);
        uint32_t r = run + upto - mine;
        while (m) {
            const int32_t slot = (int32_t)i + (__ffs((int)m) - 1);
            row_of_slot[slot] = (int32_t)r;
            slot_of_row[r] = slot;
            ++r;
            m &= m - 1;
        }
        run += (uint32_t)__builtin_amdgcn_readlane((int)upto, kWave - 1);
    };
    if (same) {  // wave-uniform
#pragma unroll
        for (int s = 0; s < kKeep; ++s)
            if (s < steps) place(base + (int64_t)s * kStep, (hits[s / 4] >> (8 * (s % 4))) & 255u);
    }
    // the last expert's workgroup, which knows the total: dropped slots and the rows past the last
    if ((int)e == E - 1 && (int64_t)total < n) {
        for (int64_t i = threadIdx.x; i < n; i += NT) {
            if ((uint32_t)ids[i] >= (uint32_t)E) row_of_slot[i] = -1;
            if (i >= (int64_t)total) slot_of_row[i] = -1;
        }
    }
}

// ---------------------------------------------------------------------------
// The same sort for many slots, where reading the list once per expert costs more
// than four launches: the list is cut into chunks of kChunkSlots (the last takes the
// rest), each workgroup counts its chunk's slots per expert, the counts are summed
// over the chunks and the experts, and each workgroup places its chunk.  The counts
// need no workspace: chunk c's lie in the first E entries of its own stretch of
// row_of_slot (E <= MXG_MAX_GROUPS <= kChunkSlots), which only the workgroup that
// reads them overwrites, in the last launch.  Four launches that wait for each other:
// 131072 slots of 128 experts 2.6, 3.2, 1.6 and 8.5 us (16 a call), in the last one 32
// workgroups whose waves take four steps one behind the other, once to count and once
// to place; 1 M slots 23 a call, past that bound by the place kernel's scattered stores.
constexpr int kChunkSlots = 4096, kSortThreads = 1024, kSortWaves = kSortThreads / kWave;
static_assert(kMaxGroups <= kChunkSlots && kMaxGroups <= kSortThreads, "a chunk holds its counts, a thread an expert");

// Counts of chunk c: LDS atomics, integers, so their order changes nothing.
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const int32_t* __restrict__ ids, int64_t n, int E,
                                                                  int32_t* __restrict__ table) {
    __shared__ uint32_t s_count[kMaxGroups];
    for (int e = threadIdx.x; e < E; e += kSortThreads) s_count[e] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * kChunkSlots;
    const int64_t hi = blockIdx.x + 1 < gridDim.x ? lo + kChunkSlots : n;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads) {
        const uint32_t id = (uint32_t)ids[i];
        if (id < (uint32_t)E) atomicAdd(&s_count[id], 1u);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kSortThreads) table[lo + e] = (int32_t)s_count[e];
}

// Running sums of an expert's counts over the chunks; its total to off[e].
// 16 experts a workgroup, 16 threads share an expert's chunks.
__global__ __launch_bounds__(kThreads) void sort_scan_kernel(int32_t* __restrict__ table, int64_t chunks, int E,
                                                             uint32_t* __restrict__ off) {
    __shared__ uint32_t s_sum[16][16];
    const int le = threadIdx.x % 16, seg = threadIdx.x / 16, e = blockIdx.x * 16 + le;
    const int64_t per = (chunks + 15) / 16, lo = seg * per, hi = lo + per < chunks ? lo + per : chunks;
    uint32_t sum = 0;
    if (e < E)
        for (int64_t c = lo; c < hi; ++c) sum += (uint32_t)table[c * kChunkSlots + e];
    s_sum[seg][le] = sum;
    __syncthreads();
    uint32_t run = 0, total = 0;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
        run += q < seg ? s_sum[q][le] : 0;
        total += s_sum[q][le];
    }
    if (e >= E) return;
    for (int64_t c = lo; c < hi; ++c) {
        const uint32_t t = (uint32_t)table[c * kChunkSlots + e];
        table[c * kChunkSlots + e] = (int32_t)run;
        run += t;
    }
    if (seg == 0) off[e] = total;
}

// The experts' totals to their offsets, in place: one workgroup.
__global__ __launch_bounds__(kSortThreads) void sort_offsets_kernel(uint32_t* __restrict__ off, int E) {
    __shared__ uint32_t s_wave[kSortWaves];
    const int e = threadIdx.x, lane = e & (kWave - 1), wave = e / kWave;
    const uint32_t mine = e < E ? off[e] : 0, upto = lane_scan(mine);
    if (lane == kWave - 1) s_wave[wave] = upto;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < wave; ++w) before += s_wave[w];
    if (e < E) off[e] = before + upto - mine;
    if (e == E - 1) off[E] = before + upto;
}

// The lanes of the wave whose id equals this one's, of the lanes that hold one.
__device__ __forceinline__ uint64_t same_id(uint32_t id, bool has, int bits) {
    uint64_t m = __ballot(has);
    for (int b = 0; b < bits; ++b) {
        const bool one = (id >> b) & 1;
        const uint64_t with = __ballot(one);
        m &= one ? with : ~with;
    }
    return m;
}

// Places chunk c.  A wave owns a contiguous stretch of it and takes 64 slots a step;
// a slot's row is its expert's offset, plus the expert's slots in the chunks and waves
// and steps before, plus the lanes before it with the same id.
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const int32_t* __restrict__ ids, int64_t n, int E,
                                                                  int bits, const uint32_t* __restrict__ off,
                                                                  int32_t* row_of_slot,
                                                                  int32_t* __restrict__ slot_of_row) {
    __shared__ uint32_t s_next[kSortWaves][kMaxGroups];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t lo = (int64_t)blockIdx.x * kChunkSlots;
    const int64_t hi = blockIdx.x + 1 < gridDim.x ? lo + kChunkSlots : n;
    for (int e = lane; e < E; e += kWave) s_next[wave][e] = 0;
    const int64_t per = ((hi - lo + kSortWaves - 1) / kSortWaves + kWave - 1) / kWave * kWave;
    const int64_t w_lo = lo + wave * per, w_hi = w_lo + per < hi ? w_lo + per : hi;
    const uint64_t below = (1ull << lane) - 1;
    auto step = [&](int64_t i0, auto use) {
        const uint32_t id = i0 + lane < w_hi ? (uint32_t)ids[i0 + lane] : ~0u;
        const bool has = id < (uint32_t)E;
        const uint64_t m = same_id(id, has, bits);
        const uint32_t next = has ? s_next[wave][id] : 0;
        use(i0 + lane, has, next + (uint32_t)__popcll(m & below));
        if (has && (m & below) == 0) s_next[wave][id] = next + (uint32_t)__popcll(m);  // the first lane of each id
    };
    for (int64_t i = w_lo; i < w_hi; i += kWave) step(i, [](int64_t, bool, uint32_t) {});
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kSortThreads) {
        uint32_t run = off[e] + (uint32_t)row_of_slot[lo + e];
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t t = s_next[w][e];
            s_next[w][e] = run;
            run += t;
        }
    }
    __syncthreads();  // the chunk's counts are read: its stretch of row_of_slot may be written
    for (int64_t i = w_lo; i < w_hi; i += kWave)
        step(i, [&](int64_t slot, bool has, uint32_t row) {
            if (slot < w_hi) row_of_slot[slot] = has ? (int32_t)row : -1;
            if (has) slot_of_row[row] = (int32_t)slot;
        });
    const int64_t total = off[E];
    for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads)
        if (i >= total) slot_of_row[i] = -1;
}

// A launch holds fewer than 2^32 threads; past this many workgroups they loop.
unsigned grid_of(int64_t blocks) { return (unsigned)(blocks < (1 << 20) ? blocks : 1 << 20); }

template <class LT, int LPT, int VPL>
hipError_t topk_as(const void* logits, const float* bias, int64_t ntok, int E, int top_k, int score, bool renorm,
                   float scale, int32_t* ids, float* weights, hipStream_t stream) {
    constexpr int kTok = kThreads / LPT;
    const dim3 grid(grid_of((ntok + kTok - 1) / kTok));
    if (bias)
        hipLaunchKernelGGL((topk_kernel<LT, LPT, VPL, true>), grid, dim3(kThreads), 0, stream,
                           static_cast<const LT*>(logits), bias, ntok, E, top_k, score, renorm, scale, ids, weights);
    else
        hipLaunchKernelGGL((topk_kernel<LT, LPT, VPL, false>), grid, dim3(kThreads), 0, stream,
                           static_cast<const LT*>(logits), bias, ntok, E, top_k, score, renorm, scale, ids, weights);
    return hipGetLastError();
}

template <class LT, int LPT, int VPL>
hipError_t topk_backward_as(const void* logits, const int32_t* ids, const float* dw, int64_t ntok, int E, int top_k,
                            int score, bool renorm, float scale, void* dlogits, hipStream_t stream) {
    constexpr int kTok = kThreads / LPT;
    hipLaunchKernelGGL((topk_backward_kernel<LT, LPT, VPL>), dim3(grid_of((ntok + kTok - 1) / kTok)),
                       dim3(kThreads), 0, stream, static_cast<const LT*>(logits), ids, dw, ntok, E, top_k, score,
                       renorm, scale, static_cast<LT*>(dlogits));
    return hipGetLastError();
}

// 16 lanes a token while they hold its experts in 16 elements and its slots in
// one each; a whole wave otherwise.  Elements no expert fills cost as much as others
// (512 experts in 8 elements a lane 11 us, in 16 16.8).
template <class LT, class F16x4, class F16x8, class F16x16, class F64x4, class F64x8, class F64x16>
hipError_t choose(int E, int top_k, F16x4 a, F16x8 b, F16x16 c, F64x4 d, F64x8 e, F64x16 f) {
    if (top_k <= 16 && E <= 64) return a();
    if (top_k <= 16 && E <= 128) return b();
    if (top_k <= 16 && E <= 256) return c();
    if (E <= 256) return d();
    return E <= 512 ? e() : f();
}

template <class LT>
hipError_t topk_type(int score, const void* lg, const float* bias, int64_t n, int E, int k, bool rn, float sc,
                     int32_t* ids, float* w, hipStream_t s) {
    return choose<LT>(
        E, k, [&] { return topk_as<LT, 16, 4>(lg, bias, n, E, k, score, rn, sc, ids, w, s); },
        [&] { return topk_as<LT, 16, 8>(lg, bias, n, E, k, score, rn, sc, ids, w, s); },
        [&] { return topk_as<LT, 16, 16>(lg, bias, n, E, k, score, rn, sc, ids, w, s); },
        [&] { return topk_as<LT, 64, 4>(lg, bias, n, E, k, score, rn, sc, ids, w, s); },
        [&] { return topk_as<LT, 64, 8>(lg, bias, n, E, k, score, rn, sc, ids, w, s); },
        [&] { return topk_as<LT, 64, 16>(lg, bias, n, E, k, score, rn, sc, ids, w, s); });
}

template <class LT>
hipError_t topk_backward_type(int score, const void* lg, const int32_t* ids, const float* dw, int64_t n, int E, int k,
                              bool rn, float sc, void* dl, hipStream_t s) {
    return choose<LT>(
        E, k, [&] { return topk_backward_as<LT, 16, 4>(lg, ids, dw, n, E, k, score, rn, sc, dl, s); },
        [&] { return topk_backward_as<LT, 16, 8>(lg, ids, dw, n, E, k, score, rn, sc, dl, s); },
        [&] { return topk_backward_as<LT, 16, 16>(lg, ids, dw, n, E, k, score, rn, sc, dl, s); },
        [&] { return topk_backward_as<LT, 64, 4>(lg, ids, dw, n, E, k, score, rn, sc, dl, s); },
        [&] { return topk_backward_as<LT, 64, 8>(lg, ids, dw, n, E, k, score, rn, sc, dl, s); },
        [&] { return topk_backward_as<LT, 64, 16>(lg, ids, dw, n, E, k, score, rn, sc, dl, s); });
}

}  // namespace

hipError_t launch_topk(int type, int score, const void* logits, const float* bias, int64_t ntok, int E, int top_k,
                       bool renorm, float scale, int32_t* ids, float* weights, hipStream_t stream) {
    return type == 0 ? topk_type<float>(score, logits, bias, ntok, E, top_k, renorm, scale, ids, weights, stream)
                     : topk_type<uint16_t>(score, logits, bias, ntok, E, top_k, renorm, scale, ids, weights, stream);
}

hipError_t launch_topk_backward(int type, int score, const void* logits, const int32_t* ids, const float* dweights,
                                int64_t ntok, int E, int top_k, bool renorm, float scale, void* dlogits,
                                hipStream_t stream) {
    return type == 0 ? topk_backward_type<float>(score, logits, ids, dweights, ntok, E, top_k, renorm, scale, dlogits,
                                                 stream)
                     : topk_backward_type<uint16_t>(score, logits, ids, dweights, ntok, E, top_k, renorm, scale,
                                                    dlogits, stream);
}

hipError_t launch_sort(const int32_t* ids, int64_t nslots, int E, uint32_t* off, int32_t* row_of_slot,
                       int32_t* slot_of_row, hipStream_t stream) {
    // The one launch reads the list once per expert, two workgroups on a CU: it wins up
    // to 65536 slots of 256 experts (8.6 us a call against 17), draws at twice that (16
    // and 16) and loses where more of either follows (16384 slots of 1024: 14 and 17,
    // 65536: 26 and 17; 1 M slots of 128: 125 and 23, of 1024: 447 and 29; 4 M of 256:
    // 490 and 66; with 97 % of 1 M slots on one expert 822 and 24).
    constexpr int64_t kOnceSlots = 65536;
    static_assert(kOnceSlots <= kKeep * 1024 * kIds, "the matches a wave keeps");
    if (nslots * (E > 256 ? E : 256) > kOnceSlots * 256) {
        const int64_t chunks = nslots / kChunkSlots;
        int bits = 0;
        while ((1 << bits) < E) ++bits;
        hipLaunchKernelGGL(sort_count_kernel, dim3((unsigned)chunks), dim3(kSortThreads), 0, stream, ids, nslots, E,
                           row_of_slot);
        hipLaunchKernelGGL(sort_scan_kernel, dim3((unsigned)((E + 15) / 16)), dim3(kThreads), 0, stream, row_of_slot,
                           chunks, E, off);
        hipLaunchKernelGGL(sort_offsets_kernel, dim3(1), dim3(kSortThreads), 0, stream, off, E);
        hipLaunchKernelGGL(sort_place_kernel, dim3((unsigned)chunks), dim3(kSortThreads), 0, stream, ids, nslots, E,
                           bits, off, row_of_slot, slot_of_row);
        return hipGetLastError();
    }
    // four waves are enough for a serving step's slots and start sooner
    if (nslots <= 4096)
        hipLaunchKernelGGL(sort_kernel<256>, dim3((unsigned)E), dim3(256), 0, stream, ids, nslots, E, off, row_of_slot,
                           slot_of_row);
    else
        hipLaunchKernelGGL(sort_kernel<1024>, dim3((unsigned)E), dim3(1024), 0, stream, ids, nslots, E, off,
                           row_of_slot, slot_of_row);
    return hipGetLastError();
}

}  // namespace mxg
