// gemm_bf16.h -- what the BF16 products' kernels share: the argument block, the
// activations with their derivatives, the epilogues of eight neighbouring columns of a
// row, and the choice of tile.  Device code for gfx950, and that choice for the host.
#pragma once

#include "mxg_device.h"
#include "mxg_internal.h"

#include <type_traits>

namespace mxg {
namespace bf16 {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

enum Act { kNone = 0, kRelu = 1, kGelu = 2, kSilu = 3, kSwiglu = 4 };  // mxg_activation

// ---------------------------------------------------------------------------
// Host side: which kernel a product of given sizes runs, by the time that each would take.
// A launch of n tiles runs in rounds of `per_cu` workgroups a CU; a round takes `base` us and,
// for each 64 of the depth that a wave has before it, `stage` us or what the workgroups'
// operands take at `rate` bytes a ns (TB/s) from the near caches, whichever is more.  Fitted to
// the times beside the candidates, of which it picks the first or one within 15 % of it (the
// sizes' own minimum, the weights from HBM, is the same for all).
struct Candidate {
    int rows, cols, waves, per_cu;  // of a tile; waves its depth is split over
    double base, stage, rate;
};
struct Work {
    int64_t groups, rows;  // that own output rows, and how many in all
    int64_t cols, depth;   // of the output, and of the sum
};
inline double time_of(const Candidate& c, const Work& w, int64_t cus) {
    // The host does not see the group sizes.  Groups of x tiles on average, uneven ones, have x + 1/2
    // each from x = 1 on (within 2 % for Zipf's law with exponents of 0.5 to 1.1), below it one and more
    // the closer x comes to 1 (5003 rows of 24: 33 of 256; 4096 of 64: 69 of 128; 512 of 8: 8).
    const double x = (double)w.rows / ((double)w.groups * c.rows), few = 1.0 + 0.7 * x * x * x;
    const int64_t some = (int64_t)((double)w.groups * (x >= 1.0 ? x + 0.5 : few < 1.5 ? few : 1.5));
    const int64_t mt = w.groups == 1 ? (w.rows + c.rows - 1) / c.rows : some;
    const int64_t nt = (w.cols + c.cols - 1) / c.cols, room = cus * c.per_cu;
    const int64_t stages = (w.depth + 63) / 64, mine = (stages + c.waves - 1) / c.waves;
    // rows and columns past the output's are not loaded
    const double tile = (double)w.rows / (double)mt + (double)w.cols / (double)nt;
    auto round = [&](double n) {
        const double near = (double)stages * tile * 128.0 * n / c.rate * 1e-6, far = (double)mine * c.stage;
        return n > 0 ? c.base + (near > far ? near : far) : 0.0;
    };
    const double tiles = (double)mt * (double)nt, whole = (double)(int64_t)(tiles / (double)room);
    return whole * round((double)room) + round(tiles - whole * (double)room);
}
template <int N>
inline int fastest(const Candidate (&c)[N], const Work& w, int64_t cus) {
    int best = 0;
    double least = time_of(c[0], w, cus);
    for (int i = 1; i < N; ++i) {
        const double t = time_of(c[i], w, cus);
        if (t < least) {
            best = i;
            least = t;
        }
    }
    return best;
}

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }
// The normal distribution's Phi(z), by erfc so that it keeps its digits where it is small.
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(z * -0.70710678118654752f); }

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == kRelu) return z < 0.0f ? 0.0f : z;  // keeps a NaN
    if constexpr (ACT == kGelu) return z * normal_cdf(z);
    if constexpr (ACT == kSilu) return z / (1.0f + expf(-z));
    return z;
}
template <int ACT>
__device__ __forceinline__ float derivative(float z) {
    if constexpr (ACT == kRelu) return z > 0.0f ? 1.0f : 0.0f;
    if constexpr (ACT == kGelu) return fmaf(z, 0.39894228040143268f * expf(-0.5f * z * z), normal_cdf(z));
    if constexpr (ACT == kSilu) {
        const float s = sigmoid(z);
        return s * (1.0f + z * (1.0f - s));
    }
    return 1.0f;
}
// Runs f with the activation as a constant.
template <class F>
__device__ __forceinline__ void with_act(int act, F f) {
    switch (act) {
        case kRelu: f(std::integral_constant<int, kRelu>{}); break;
        case kGelu: f(std::integral_constant<int, kGelu>{}); break;
        case kSilu: f(std::integral_constant<int, kSilu>{}); break;
        case kSwiglu: f(std::integral_constant<int, kSwiglu>{}); break;
        default: f(std::integral_constant<int, kNone>{}); break;
    }
}

// W neighbouring elements at p (fp32 or bf16): whole (aligned to W elements, 16 bytes at most),
// or the first n.  Whole ones are stored with the nontemporal hint (8192^3 753 -> 729 us, 32768 rows
// of 64 experts, 1536 x 4096, fp32 weights' gradient 861 -> 793).
template <int W>
__device__ __forceinline__ void load_n(const void* p, bool f32, bool whole, int n, float* v) {
    if (f32) {
        const float* q = static_cast<const float*>(p);
        constexpr int V = W < 4 ? W : 4;
        typedef float vt __attribute__((ext_vector_type(V)));
        if (whole) {
#pragma unroll
            for (int i = 0; i < W; i += V) {
                const vt x = *reinterpret_cast<const vt*>(q + i);
#pragma unroll
                for (int j = 0; j < V; ++j) v[i + j] = x[j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) v[i] = i < n ? q[i] : 0.0f;
        }
    } else {
        const uint16_t* q = static_cast<const uint16_t*>(p);
        constexpr int V = W < 8 ? W : 8;
        typedef uint16_t vt __attribute__((ext_vector_type(V)));
        if (whole) {
#pragma unroll
            for (int i = 0; i < W; i += V) {
                const vt x = *reinterpret_cast<const vt*>(q + i);
#pragma unroll
                for (int j = 0; j < V; ++j) v[i + j] = bf16_to_f32(x[j]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) v[i] = i < n ? bf16_to_f32(q[i]) : 0.0f;
        }
    }
}
template <int W>
__device__ __forceinline__ void store_n(void* p, bool f32, bool whole, int n, const float* v) {
    if (f32) {
        float* q = static_cast<float*>(p);
        constexpr int V = W < 4 ? W : 4;
        typedef float vt __attribute__((ext_vector_type(V)));
        if (whole) {
#pragma unroll
            for (int i = 0; i < W; i += V) {
                vt x;
#pragma unroll
                for (int j = 0; j < V; ++j) x[j] = v[i + j];
                __builtin_nontemporal_store(x, reinterpret_cast<vt*>(q + i));
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
                if (i < n) q[i] = v[i];
        }
    } else {
        uint16_t* q = static_cast<uint16_t*>(p);
        constexpr int V = W < 8 ? W / 2 : 4;
        typedef uint32_t vt __attribute__((ext_vector_type(V)));
        if (whole) {
#pragma unroll
            for (int i = 0; i < W; i += 2 * V) {
                vt x;
#pragma unroll
                for (int j = 0; j < V; ++j) x[j] = f32x2_to_bf16x2(v[i + 2 * j], v[i + 2 * j + 1]);
                __builtin_nontemporal_store(x, reinterpret_cast<vt*>(q + i));
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
                if (i < n) q[i] = (uint16_t)f32_to_bf16(v[i]);
        }
    }
}

// The forward epilogue of columns col .. col + 7 of row t of expert e, from the sums v: what it
// reads beside them, asked for ahead, and the rest.  WHOLE: N is a multiple of 8, else only the
// columns below N count.
struct Beside {
    float bias[8], res[8];
};
template <int ACT, bool WHOLE>
__device__ __forceinline__ void fetch8(const Bf16Problem& p, int e, int64_t t, int64_t col, Beside& x) {
    const int n = WHOLE || p.N - col > 8 ? 8 : (int)(p.N - col);
    if (p.bias) load_n<8>(p.bias + e * p.N + col, true, WHOLE && p.bias16, n, x.bias);
    if (!p.res) return;
    const int size = p.c32 ? 4 : 2;
    if constexpr (ACT == kSwiglu)
        load_n<4>(static_cast<const uint8_t*>(p.res) + (t * (p.N / 2) + col / 2) * size, p.c32, WHOLE, n / 2, x.res);
    else load_n<8>(static_cast<const uint8_t*>(p.res) + (t * p.N + col) * size, p.c32, WHOLE, n, x.res);
}
template <int ACT, bool WHOLE>
__device__ __forceinline__ void finish8(const Bf16Problem& p, int64_t t, int64_t col, const float* sums,
                                        const Beside& x) {
    const int n = WHOLE || p.N - col > 8 ? 8 : (int)(p.N - col);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p.bias ? sums[i] + x.bias[i] : sums[i];
    if (p.z) store_n<8>(static_cast<uint16_t*>(p.z) + t * p.N + col, false, WHOLE, n, v);
    const int size = p.c32 ? 4 : 2;
    if constexpr (ACT == kSwiglu) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[i] = activate<kSilu>(v[2 * i]) * v[2 * i + 1];
            if (p.res) y[i] += x.res[i];
        }
        store_n<4>(static_cast<uint8_t*>(p.c) + (t * (p.N / 2) + col / 2) * size, p.c32, WHOLE, n / 2, y);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = activate<ACT>(v[i]);
            if (p.res) v[i] += x.res[i];
        }
        store_n<8>(static_cast<uint8_t*>(p.c) + (t * p.N + col) * size, p.c32, WHOLE, n, v);
    }
}

// d times the derivative at z: the gate and up columns of N sums.
template <int N>
__device__ __forceinline__ void swiglu_grad(const float* z, const float* d, float* out) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float g = z[2 * i], u = z[2 * i + 1], s = sigmoid(g);
        out[2 * i] = d[i] * u * s * (1.0f + g * (1.0f - s));
        out[2 * i + 1] = d[i] * g * s;
    }
}

// The backward epilogue of W columns of row t (K is a multiple of 8): the
// pre-activations, asked for ahead, and the rest.
template <int W>
struct Before {
    float z[2 * W];
};
template <int ACT, int W>
__device__ __forceinline__ void fetch_backward(const Bf16Problem& p, int64_t t, int64_t col, Before<W>& x) {
    if constexpr (ACT == kSwiglu)
        load_n<2 * W>(static_cast<const uint16_t*>(p.z) + (t * p.K + col) * 2, false, true, 2 * W, x.z);
    else if constexpr (ACT != kNone)
        load_n<W>(static_cast<const uint16_t*>(p.z) + t * p.K + col, false, true, W, x.z);
}
template <int ACT, int W>
__device__ __forceinline__ void finish_backward(const Bf16Problem& p, int64_t t, int64_t col, const float* d,
                                                const Before<W>& x) {
    if constexpr (ACT == kSwiglu) {
        float out[2 * W];
        swiglu_grad<W>(x.z, d, out);
        store_n<2 * W>(static_cast<uint16_t*>(p.c) + (t * p.K + col) * 2, false, true, 2 * W, out);
    } else {
        float v[W];
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = ACT == kNone ? d[i] : d[i] * derivative<ACT>(x.z[i]);
        store_n<W>(static_cast<uint16_t*>(p.c) + t * p.K + col, false, true, W, v);
    }
}

}  // namespace bf16
}  // namespace mxg
