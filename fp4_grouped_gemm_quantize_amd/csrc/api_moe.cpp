// api_moe.cpp -- the extern "C" entry points of the router, the routing plan,
// the 128-block FP8 format and their gradients: argument validation on the
// host (before anything is enqueued), then one launch (a long sort: four).  No
// allocation outside the MXG_VALIDATE check, no host synchronisation outside
// it, no state.  No exception leaves an entry point.
#include "api_common.h"

using namespace mxg::api;

namespace {

bool valid_type(int t) { return t == MXG_F32 || t == MXG_BF16; }
bool valid_score(int s) { return s == MXG_SCORE_SOFTMAX || s == MXG_SCORE_SIGMOID; }
uintptr_t type_bytes(int t) { return t == MXG_F32 ? 4 : 2; }

// With MXG_VALIDATE set: refuse a row_of_slot that names a row twice (the entry
// points that write rows through it).  The rows are [0, T), or with off those that
// its G groups cover: [off[0], off[G]), since check_routing has seen that the offsets
// rise and stay within T.
mxg_status check_distinct_rows(const int32_t* row_of_slot, int64_t nslots, int64_t T, hipStream_t stream,
                               const uint32_t* off = nullptr, int32_t G = 0) {
    if (!validation_on()) return MXG_SUCCESS;
    t_validation_msg[0] = '\0';
    try {
        std::vector<int32_t> h((size_t)nslots);
        uint32_t ends[2] = {0, 0};
        if (hipMemcpyAsync(h.data(), row_of_slot, sizeof(int32_t) * h.size(), hipMemcpyDeviceToHost, stream) !=
                hipSuccess ||
            (off != nullptr &&
             (hipMemcpyAsync(&ends[0], off, sizeof ends[0], hipMemcpyDeviceToHost, stream) != hipSuccess ||
              hipMemcpyAsync(&ends[1], off + G, sizeof ends[1], hipMemcpyDeviceToHost, stream) != hipSuccess)) ||
            hipStreamSynchronize(stream) != hipSuccess)
            return MXG_ERROR_LAUNCH;
        const int64_t lo = off != nullptr ? ends[0] : 0, hi = off != nullptr ? (int64_t)ends[1] : T;
        std::vector<bool> seen((size_t)(hi < INT32_MAX ? hi : (int64_t)INT32_MAX + 1));  // what an int32 can name
        for (int64_t i = 0; i < nslots; ++i) {
            const int64_t r = h[(size_t)i];
            if (r < lo || r >= hi) continue;
            if (seen[(size_t)r]) {
                snprintf(t_validation_msg, sizeof t_validation_msg, "row_of_slot[%lld] = %lld names a row again",
                         (long long)i, (long long)r);
                return MXG_ERROR_INVALID_VALUE;
            }
            seen[(size_t)r] = true;
        }
    } catch (const std::exception&) {
        return MXG_ERROR_LAUNCH;
    }
    return MXG_SUCCESS;
}

mxg_status check_topk_sizes(int type, int score, int64_t ntok, int32_t E, int32_t top_k) {
    if (!valid_type(type) || !valid_score(score)) return MXG_ERROR_INVALID_VALUE;
    if (ntok < 0 || E < 1 || top_k < 1) return MXG_ERROR_INVALID_VALUE;
    if (E > MXG_MAX_GROUPS || top_k > 64 || ntok > INT32_MAX / top_k) return MXG_ERROR_NOT_SUPPORTED;
    return MXG_SUCCESS;
}

mxg_status check_rows_sizes(int64_t T, int64_t H, int64_t ntok, int32_t top_k) {
    if (H <= 0 || T < 0 || ntok < 0 || top_k < 1) return MXG_ERROR_INVALID_VALUE;
    if (H % 8 != 0 || H > INT32_MAX || ntok > INT32_MAX / top_k) return MXG_ERROR_NOT_SUPPORTED;
    return MXG_SUCCESS;
}

mxg_status check_quantize_sizes(int64_t K, int64_t T, int32_t G) {
    if (K <= 0 || T < 0 || G < 0) return MXG_ERROR_INVALID_VALUE;
    if (K % 32 != 0 || K > INT32_MAX / 2 || T > INT32_MAX || G > MXG_MAX_GROUPS) return MXG_ERROR_NOT_SUPPORTED;
    return MXG_SUCCESS;
}

}  // namespace

extern "C" {

mxg_status mx_moe_topk(mxg_dtype logits_type, mxg_score score, const void* logits, const float* bias,
                       int64_t num_tokens, int32_t num_experts, int32_t top_k, int32_t renormalize, float scale,
                       int32_t* topk_ids, float* topk_weights, hipStream_t stream) {
    if (mxg_status st = check_topk_sizes(logits_type, score, num_tokens, num_experts, top_k)) return st;
    if (top_k > num_experts) return MXG_ERROR_NOT_SUPPORTED;
    if (num_tokens == 0) return MXG_SUCCESS;  // nothing is read or written
    if (!logits || !topk_ids || !topk_weights) return MXG_ERROR_INVALID_VALUE;
    if (!aligned(logits, type_bytes(logits_type)) || !aligned(bias, 4) || !aligned(topk_ids, 4) ||
        !aligned(topk_weights, 4))
        return MXG_ERROR_INVALID_VALUE;
    return from_hip(mxg::launch_topk((int)logits_type, (int)score, logits, bias, num_tokens, num_experts, top_k,
                                     renormalize != 0, scale, topk_ids, topk_weights, stream));
}

mxg_status mx_moe_topk_backward(mxg_dtype logits_type, mxg_score score, const void* logits, const int32_t* topk_ids,
                                const float* dweights, int64_t num_tokens, int32_t num_experts, int32_t top_k,
                                int32_t renormalize, float scale, void* dlogits, hipStream_t stream) {
    if (mxg_status st = check_topk_sizes(logits_type, score, num_tokens, num_experts, top_k)) return st;
    if (num_tokens == 0) return MXG_SUCCESS;  // nothing is read or written
    if (!logits || !topk_ids || !dweights || !dlogits) return MXG_ERROR_INVALID_VALUE;
    if (!aligned(logits, type_bytes(logits_type)) || !aligned(dlogits, type_bytes(logits_type)) ||
        !aligned(topk_ids, 4) || !aligned(dweights, 4))
        return MXG_ERROR_INVALID_VALUE;
    return from_hip(mxg::launch_topk_backward((int)logits_type, (int)score, logits, topk_ids, dweights, num_tokens,
                                              num_experts, top_k, renormalize != 0, scale, dlogits, stream));
}

mxg_status mx_moe_sort(const int32_t* topk_ids, int64_t num_tokens, int32_t top_k, int32_t num_experts,
                       uint32_t* row_offsets, int32_t* row_of_slot, int32_t* slot_of_row, hipStream_t stream) {
    if (num_tokens < 0 || top_k < 1 || num_experts < 1) return MXG_ERROR_INVALID_VALUE;
    if (num_experts > MXG_MAX_GROUPS || num_tokens > INT32_MAX / top_k) return MXG_ERROR_NOT_SUPPORTED;
    if (!row_offsets || !aligned(row_offsets, 4)) return MXG_ERROR_INVALID_VALUE;
    if (num_tokens > 0 && (!topk_ids || !row_of_slot || !slot_of_row || !aligned(topk_ids, 4) ||
                           !aligned(row_of_slot, 4) || !aligned(slot_of_row, 4)))
        return MXG_ERROR_INVALID_VALUE;
    return from_hip(mxg::launch_sort(topk_ids, num_tokens * top_k, num_experts, row_offsets, row_of_slot, slot_of_row,
                                     stream));
}

mxg_status mx_moe_permute(const void* x_bf16, int64_t num_tokens, int64_t H, const int32_t* row_of_slot,
                          int32_t top_k, void* rows_bf16, int64_t total_rows, hipStream_t stream) {
    if (mxg_status st = check_rows_sizes(total_rows, H, num_tokens, top_k)) return st;
    if (num_tokens == 0) return MXG_SUCCESS;  // nothing is read or written
    if (!x_bf16 || !row_of_slot || (total_rows > 0 && !rows_bf16)) return MXG_ERROR_INVALID_VALUE;
    if (!aligned(x_bf16, 16) || !aligned(rows_bf16, 16) || !aligned(row_of_slot, 4)) return MXG_ERROR_INVALID_VALUE;
    if (total_rows == 0) return MXG_SUCCESS;
    if (mxg_status st = check_distinct_rows(row_of_slot, num_tokens * top_k, total_rows, stream)) return st;
    return from_hip(mxg::launch_permute(x_bf16, num_tokens, H, row_of_slot, top_k, rows_bf16, total_rows, stream));
}

mxg_status mx_moe_permute_backward(const void* drows_bf16, int64_t total_rows, int64_t H, const int32_t* row_of_slot,
                                   int64_t num_tokens, int32_t top_k, void* dx_bf16, hipStream_t stream) {
    if (mxg_status st = check_rows_sizes(total_rows, H, num_tokens, top_k)) return st;
    if (num_tokens == 0) return MXG_SUCCESS;  // nothing is read or written
    if (!dx_bf16 || !row_of_slot || (total_rows > 0 && !drows_bf16)) return MXG_ERROR_INVALID_VALUE;
    if (!aligned(drows_bf16, 16) || !aligned(dx_bf16, 16) || !aligned(row_of_slot, 4)) return MXG_ERROR_INVALID_VALUE;
    return from_hip(mxg::launch_permute_backward(drows_bf16, total_rows, H, row_of_slot, num_tokens, top_k, dx_bf16,
                                                 stream));
}

mxg_status mx_moe_combine_backward(const void* dout_bf16, const void* y_bf16, int64_t total_rows, int64_t H,
                                   const int32_t* row_of_slot, const float* weights, int64_t num_tokens,
                                   int32_t top_k, void* dy_bf16, float* dweights, hipStream_t stream) {
    if (mxg_status st = check_rows_sizes(total_rows, H, num_tokens, top_k)) return st;
    if (num_tokens == 0) return MXG_SUCCESS;  // nothing is read or written
    if (!dout_bf16 || !row_of_slot || !weights || !dweights || (total_rows > 0 && (!y_bf16 || !dy_bf16)))
        return MXG_ERROR_INVALID_VALUE;
    if (!aligned(dout_bf16, 16) || !aligned(y_bf16, 16) || !aligned(dy_bf16, 16) || !aligned(row_of_slot, 4) ||
        !aligned(weights, 4) || !aligned(dweights, 4))
        return MXG_ERROR_INVALID_VALUE;
    if (mxg_status st = check_distinct_rows(row_of_slot, num_tokens * top_k, total_rows, stream)) return st;
    return from_hip(mxg::launch_combine_backward(dout_bf16, y_bf16, total_rows, H, row_of_slot, weights, num_tokens,
                                                 top_k, dy_bf16, dweights, stream));
}

mxg_status mx_grouped_quantize_block128(const void* x_bf16, void* q, float* scales, const uint32_t* row_offsets,
                                        int32_t num_groups, int64_t total_rows, int64_t K, hipStream_t stream) {
    if (mxg_status st = check_quantize_sizes(K, total_rows, num_groups)) return st;
    if (total_rows == 0 || num_groups == 0) return MXG_SUCCESS;  // nothing is read or written
    if (!x_bf16 || !q || !scales || !row_offsets) return MXG_ERROR_INVALID_VALUE;
    if (!aligned(x_bf16, 16) || !aligned(q, 16) || !aligned(scales, 4) || !aligned(row_offsets, 4))
        return MXG_ERROR_INVALID_VALUE;
    if (mxg_status st = check_routing(row_offsets, nullptr, num_groups, 0, total_rows, stream)) return st;
    return from_hip(mxg::launch_quantize_block128(x_bf16, total_rows, nullptr, 1, q, scales, row_offsets, num_groups,
                                                  total_rows, K, stream));
}

mxg_status mx_grouped_quantize_block128_scatter(const void* x_tokens, int64_t num_tokens, const int32_t* row_of_slot,
                                                int32_t top_k, void* q, float* scales, const uint32_t* row_offsets,
                                                int32_t num_groups, int64_t total_rows, int64_t K,
                                                hipStream_t stream) {
    if (mxg_status st = check_quantize_sizes(K, total_rows, num_groups)) return st;
    if (num_tokens < 0 || top_k < 1) return MXG_ERROR_INVALID_VALUE;
    if (top_k > 64 || num_tokens > INT32_MAX / top_k) return MXG_ERROR_NOT_SUPPORTED;
    if (total_rows == 0 || num_groups == 0 || num_tokens == 0) return MXG_SUCCESS;  // nothing is read or written
    if (!x_tokens || !row_of_slot || !q || !scales || !row_offsets) return MXG_ERROR_INVALID_VALUE;
    if (!aligned(x_tokens, 16) || !aligned(q, 16) || !aligned(scales, 4) || !aligned(row_offsets, 4) ||
        !aligned(row_of_slot, 4))
        return MXG_ERROR_INVALID_VALUE;
    if (mxg_status st = check_routing(row_offsets, nullptr, num_groups, 0, total_rows, stream)) return st;
    if (mxg_status st = check_distinct_rows(row_of_slot, num_tokens * top_k, total_rows, stream, row_offsets,
                                            num_groups))
        return st;
    return from_hip(mxg::launch_quantize_block128(x_tokens, num_tokens, row_of_slot, top_k, q, scales, row_offsets,
                                                  num_groups, total_rows, K, stream));
}

mxg_status mx_quantize_weights_block128(const void* w_bf16, int32_t num_experts, int64_t N, int64_t K, void* q,
                                        float* scales, void* q_t, float* scales_t, hipStream_t stream) {
    if (num_experts <= 0 || N <= 0 || K <= 0) return MXG_ERROR_INVALID_VALUE;
    if ((q_t == nullptr) != (scales_t == nullptr)) return MXG_ERROR_INVALID_VALUE;
    if (K % 32 != 0 || (q_t && N % 32 != 0) || N > INT32_MAX / 2 || K > INT32_MAX / 2) return MXG_ERROR_NOT_SUPPORTED;
    if (!w_bf16 || !q || !scales) return MXG_ERROR_INVALID_VALUE;
    if (!aligned(w_bf16, 16) || !aligned(q, 16) || !aligned(scales, 4) || !aligned(q_t, 16) || !aligned(scales_t, 4))
        return MXG_ERROR_INVALID_VALUE;
    return from_hip(mxg::launch_quantize_weights_block128(w_bf16, num_experts, N, K, q, scales, q_t, scales_t, stream));
}

mxg_status mx_grouped_matmul_block128(const void* a_q, const float* a_scales, const void* b_q, const float* b_scales,
                                      void* c_bf16, const uint32_t* row_offsets, const int32_t* expert_ids,
                                      int32_t num_groups, int32_t num_experts, int64_t total_rows, int64_t N,
                                      int64_t K, int64_t max_rows_per_group_hint, hipStream_t stream) {
    if (K <= 0 || N <= 0 || num_experts <= 0 || total_rows < 0 || num_groups < 0) return MXG_ERROR_INVALID_VALUE;
    if (K % 32 != 0 || K > MXG_MAX_K || num_groups > MXG_MAX_GROUPS) return MXG_ERROR_NOT_SUPPORTED;
    if (N > INT32_MAX / 2 || total_rows > INT32_MAX) return MXG_ERROR_NOT_SUPPORTED;
    if (total_rows == 0 || num_groups == 0) return MXG_SUCCESS;  // nothing is read or written
    if (!a_q || !a_scales || !b_q || !b_scales || !c_bf16 || !row_offsets || !expert_ids)
        return MXG_ERROR_INVALID_VALUE;
    if (!aligned(a_q, 16) || !aligned(b_q, 16) || !aligned(c_bf16, 16) || !aligned(a_scales, 4) ||
        !aligned(b_scales, 4) || !aligned(row_offsets, 4) || !aligned(expert_ids, 4))
        return MXG_ERROR_INVALID_VALUE;
    if (mxg_status st = check_routing(row_offsets, expert_ids, num_groups, num_experts, total_rows, stream)) return st;
    mxg::GemmProblem p{0, a_q, a_scales, b_q, b_scales, c_bf16, nullptr, nullptr, row_offsets, expert_ids,
                       num_groups, num_experts, total_rows, N, K, max_rows_per_group_hint};
    return from_hip(mxg::launch_grouped_gemm_block128(p, stream));
}

mxg_status mx_silu_quantize_block128(const void* h_bf16, void* y_q, float* y_scales, const uint32_t* row_offsets,
                                     int32_t num_groups, int64_t total_rows, int64_t I, hipStream_t stream) {
    if (mxg_status st = check_quantize_sizes(I, total_rows, num_groups)) return st;
    if (I > INT32_MAX / 4) return MXG_ERROR_NOT_SUPPORTED;
    if (total_rows == 0 || num_groups == 0) return MXG_SUCCESS;  // nothing is read or written
    if (!h_bf16 || !y_q || !y_scales || !row_offsets) return MXG_ERROR_INVALID_VALUE;
    if (!aligned(h_bf16, 16) || !aligned(y_q, 16) || !aligned(y_scales, 4) || !aligned(row_offsets, 4))
        return MXG_ERROR_INVALID_VALUE;
    if (mxg_status st = check_routing(row_offsets, nullptr, num_groups, 0, total_rows, stream)) return st;
    return from_hip(mxg::launch_silu_quantize_block128(h_bf16, y_q, y_scales, row_offsets, num_groups, total_rows, I,
                                                       stream));
}

mxg_status mx_silu_backward_block128(const void* h_bf16, const void* dy_bf16, void* dh_bf16, void* dh_q,
                                     float* dh_scales, const uint32_t* row_offsets, int32_t num_groups,
                                     int64_t total_rows, int64_t I, hipStream_t stream) {
    if (mxg_status st = check_quantize_sizes(I, total_rows, num_groups)) return st;
    if (I > INT32_MAX / 4) return MXG_ERROR_NOT_SUPPORTED;
    if (total_rows == 0 || num_groups == 0) return MXG_SUCCESS;  // nothing is read or written
    if ((dh_q == nullptr) != (dh_scales == nullptr) || (!dh_bf16 && !dh_q)) return MXG_ERROR_INVALID_VALUE;
    if (!h_bf16 || !dy_bf16 || !row_offsets) return MXG_ERROR_INVALID_VALUE;
    if (!aligned(h_bf16, 16) || !aligned(dy_bf16, 16) || !aligned(dh_bf16, 16) || !aligned(dh_q, 16) ||
        !aligned(dh_scales, 4) || !aligned(row_offsets, 4))
        return MXG_ERROR_INVALID_VALUE;
    if (mxg_status st = check_routing(row_offsets, nullptr, num_groups, 0, total_rows, stream)) return st;
    return from_hip(mxg::launch_silu_backward_block128(h_bf16, dy_bf16, dh_bf16, dh_q, dh_scales, row_offsets,
                                                       num_groups, total_rows, I, stream));
}

}  // extern "C"
