// mxg_internal.h -- launchers the C ABI layer calls; host-side only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxg {

hipError_t launch_quantize(int fmt, const void* x, void* q, void* scales, const uint32_t* off, int G, int64_t T,
                           int64_t K, hipStream_t stream);

// The same with row t read from row indices[t] / divisor of x (nsrc rows).
hipError_t launch_quantize_gather(int fmt, const void* x, int64_t nsrc, const int32_t* indices, int32_t divisor,
                                  void* q, void* scales, const uint32_t* off, int G, int64_t T, int64_t K,
                                  hipStream_t stream);

// Token-major form: token row s (of ntok) is quantized once into every routed row
// row_of_slot[s * top_k + k] in [0, T) that a group covers (top_k <= 64; FP8 rowwise K <= 8192).
hipError_t launch_quantize_scatter(int fmt, const void* x, int64_t ntok, const int32_t* row_of_slot, int top_k,
                                   void* q, void* scales, const uint32_t* off, int G, int64_t T, int64_t K,
                                   hipStream_t stream);

// MX (fmt 1, 2) with group g's scales from row scales_offsets[g] of a [scale_rows, K/32] tensor.
hipError_t launch_quantize_padded(int fmt, const void* x, void* q, void* scales, const uint32_t* scales_offsets,
                                  int64_t scale_rows, const uint32_t* off, int G, int64_t T, int64_t K,
                                  hipStream_t stream);

// NVFP4: rows of group g use tensor_scales[ids[g]]; groups with an id outside [0, E) are skipped.
hipError_t launch_quantize_nvfp4(const void* x, void* q, void* scales, const float* tensor_scales,
                                  const uint32_t* off, const int32_t* ids, int G, int E, int64_t T, int64_t K,
                                  hipStream_t stream);

// NVFP4 with group g's E4M3 scales from row scales_offsets[g] of a [scale_rows, K/16] tensor.
hipError_t launch_quantize_nvfp4_padded(const void* x, void* q, void* scales, const float* tensor_scales,
                                        const uint32_t* scales_offsets, int64_t scale_rows, const uint32_t* off,
                                        const int32_t* ids, int G, int E, int64_t T, int64_t K, hipStream_t stream);

// out[t, :] = bf16(sum_k weights[t*top_k + k] * y[row_of_slot[t*top_k + k], :]).
hipError_t launch_combine(const void* y, int64_t T, int64_t H, const int32_t* row_of_slot, const float* weights,
                          int64_t ntok, int top_k, void* out, hipStream_t stream);

hipError_t launch_silu_quantize(const void* h, void* yq, void* ys, const uint32_t* off, int G, int64_t T,
                                int64_t I, hipStream_t stream);

// NVFP4 requant of y = bf16(silu(g) u): rows of group g use y_scales_sf[ids[g]].
hipError_t launch_silu_quantize_nvfp4(const void* h, void* yq, void* ys, const float* y_sf, const uint32_t* off,
                                      const int32_t* ids, int G, int E, int64_t T, int64_t I, hipStream_t stream);

// Grouped GEMM; when yq != nullptr the SwiGLU + MXFP4 requant epilogue runs
// (N = 2I) and c is not written.
struct GemmProblem {
    int fmt;
    const void* a;
    const void* a_scales;
    const void* b;
    const void* b_scales;
    void* c;
    void* yq;
    void* ys;
    const uint32_t* off;
    const int32_t* ids;
    int G;
    int E;
    int64_t T;
    int64_t N;
    int64_t K;
    int64_t max_rows_hint;
    const float* es;   // NVFP4 (fmt 3): per-expert epilogue scale, fp32 [E]
    const void* rs;    // NVFP4 fused: optional bf16 row scales [T]
    const float* ysf;  // NVFP4 fused: per-expert encode-side tensor scale of y, fp32 [E]
    const uint32_t* asoff;  // padded A scales: group g's rows from row asoff[g] (nullptr: dense)
    int64_t as_rows;        // rows of that scale tensor
    bool b_prepared;        // FP8 rowwise: b holds the prepared weights (launch_prepare_weights)
};

hipError_t launch_grouped_gemm(const GemmProblem& p, hipStream_t stream);

// The FP8 rowwise tile launch_grouped_gemm runs for p: 384 or 256 (256-row
// tiles of that many columns), 32 (the 32 x 256 decode tile), 0 otherwise.
int fp8_tile_choice(const GemmProblem& p);

// FP8 rowwise weights [E, N, K] (K a multiple of 64) into the layout the
// GEMM's 64-byte-stage rings load as it is; out holds prepared_weights_bytes(E, N, K).
int64_t prepared_weights_bytes(int64_t E, int64_t N, int64_t K);
hipError_t launch_prepare_weights(const void* b, int64_t E, int64_t N, int64_t K, void* out, hipStream_t stream);

// The router and the routing plan (route.hip).  type: 0 fp32, 1 bf16 logits; score: 0 softmax, 1 sigmoid.
hipError_t launch_topk(int type, int score, const void* logits, const float* bias, int64_t ntok, int E, int top_k,
                       bool renorm, float scale, int32_t* ids, float* weights, hipStream_t stream);
hipError_t launch_topk_backward(int type, int score, const void* logits, const int32_t* ids, const float* dweights,
                                int64_t ntok, int E, int top_k, bool renorm, float scale, void* dlogits,
                                hipStream_t stream);
hipError_t launch_sort(const int32_t* ids, int64_t nslots, int E, uint32_t* off, int32_t* row_of_slot,
                       int32_t* slot_of_row, hipStream_t stream);

// Rows into expert order and the gradients of the way there and back (combine.hip).
hipError_t launch_permute(const void* x, int64_t ntok, int64_t H, const int32_t* row_of_slot, int top_k, void* rows,
                          int64_t T, hipStream_t stream);
hipError_t launch_permute_backward(const void* drows, int64_t T, int64_t H, const int32_t* row_of_slot, int64_t ntok,
                                   int top_k, void* dx, hipStream_t stream);
hipError_t launch_combine_backward(const void* dout, const void* y, int64_t T, int64_t H, const int32_t* row_of_slot,
                                   const float* weights, int64_t ntok, int top_k, void* dy, float* dweights,
                                   hipStream_t stream);

// FP8 with 128-element block scales (block128.hip, gemm_block128.hip).  row_of_slot == nullptr: row-major, x has T rows.
hipError_t launch_quantize_block128(const void* x, int64_t ntok, const int32_t* row_of_slot, int top_k, void* q,
                                    float* scales, const uint32_t* off, int G, int64_t T, int64_t K,
                                    hipStream_t stream);
hipError_t launch_quantize_weights_block128(const void* w, int64_t E, int64_t N, int64_t K, void* q, float* scales,
                                            void* q_t, float* scales_t, hipStream_t stream);
hipError_t launch_silu_quantize_block128(const void* h, void* yq, float* ys, const uint32_t* off, int G, int64_t T,
                                         int64_t I, hipStream_t stream);
hipError_t launch_silu_backward_block128(const void* h, const void* dy, void* dh, void* dh_q, float* dh_scales,
                                         const uint32_t* off, int G, int64_t T, int64_t I, hipStream_t stream);
hipError_t launch_grouped_gemm_block128(const GemmProblem& p, hipStream_t stream);
// Rows a tile of the kernel it runs for these sizes: 256, 128, 32, 16 (the row kernel), 0 (nothing).
int block128_tile_choice(const GemmProblem& p);

// Workgroups of `threads` for n units of work.  A launch holds fewer than 2^32 threads; past 2^28 of them, 512 times
// what a device runs at once, the workgroups loop.
inline unsigned workgroups(int64_t n, int threads) {
    const int64_t most = (int64_t{1} << 28) / threads;
    return (unsigned)(n < most ? n : most);
}

// The norm of a residual stream and its gradient (norm.hip).  fmt: mxg_norm_format; s32, w32: fp32 stream, weight.
hipError_t launch_rmsnorm(int fmt, bool s32, const void* x, const void* res, bool w32, const void* w, float w_add,
                          float eps, int64_t T, int64_t H, void* h, void* y, void* q, void* scales,
                          hipStream_t stream);
int64_t rmsnorm_workspace_rows(int64_t T, int64_t H);  // of H floats each
hipError_t launch_rmsnorm_backward(bool s32, const void* dy, const void* h, bool w32, const void* w, float w_add,
                                   float eps, const void* dh, int64_t T, int64_t H, void* dx, void* dx_bf16,
                                   float* dw, float* ws, hipStream_t stream);

// BF16 products and their gradients (gemm_bf16.hip, gemm_bf16_weights.hip).  off == nullptr (with ids): one group
// of all T rows, expert 0.  act: mxg_activation.
struct Bf16Problem {
    int act;
    const void* a;      // [T, K]; backward: dc [T, N]
    const void* b;      // [E, N, K]
    const float* bias;  // [E, N] or nullptr
    const void* res;    // as c, or nullptr
    void* c;            // backward: da
    bool c32;           // c and res in fp32
    void* z;            // forward: kept pre-activations or nullptr; backward: those of act
    const uint32_t* off;
    const int32_t* ids;
    int G;
    int E;
    int64_t T;
    int64_t N;
    int64_t K;
    int64_t max_rows_hint;
    bool bias16;        // bias lies on 16 bytes
};
hipError_t launch_matmul_bf16(const Bf16Problem& p, hipStream_t stream);
hipError_t launch_matmul_bf16_backward(const Bf16Problem& p, hipStream_t stream);
hipError_t launch_matmul_bf16_weights(const void* dc, const void* a, void* dw, bool dw32, float* dbias,
                                      bool accumulate, const uint32_t* off, const int32_t* ids, int G, int E,
                                      int64_t T, int64_t N, int64_t K, hipStream_t stream);
// 1000 * rows + columns of a tile of the kernel that a product, its rows' gradient (back) or its weights' gradient of these sizes runs.
int bf16_tile_choice(const Bf16Problem& p, bool back);
int bf16_weights_tile_choice(int G, int E, int64_t T, int64_t N, int64_t K);
hipError_t launch_activation_backward(int act, const void* dc, const void* z, void* dz, int64_t T, int64_t N,
                                      hipStream_t stream);

// One wave: out[0] = shader-clock ticks, out[1] = 100 MHz ticks (>= ticks) of one sleep window.
hipError_t launch_clock_probe(unsigned long long* out, unsigned long long ticks, hipStream_t stream);

}  // namespace mxg
