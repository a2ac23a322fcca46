// api_dense.cpp -- the extern "C" entry points of the norm, the BF16 products with
// their epilogue, and the gradients of both: argument validation on the host (before
// anything is enqueued), then one launch (the norm's weight gradient: two).  No
// allocation or host synchronisation outside the MXG_VALIDATE check, no state.  No
// exception leaves an entry point.
#include "api_common.h"

#include <initializer_list>

using namespace mxg::api;

namespace {

// A tensor's bytes (nullptr: none), of up to three sizes and elements of `size` bytes; sizes that no
// memory holds end at the largest number.
struct Span {
    uintptr_t lo, hi;
    Span(const void* p, uint64_t size, uint64_t a, uint64_t b = 1, uint64_t c = 1) : lo((uintptr_t)p) {
        uint64_t n = 0;
        if (p == nullptr) n = 0;
        else if (__builtin_mul_overflow(a, b, &n) || __builtin_mul_overflow(n, c, &n) ||
                 __builtin_mul_overflow(n, size, &n))
            n = UINT64_MAX;
        if (__builtin_add_overflow(lo, (uintptr_t)n, &hi)) hi = UINTPTR_MAX;
    }
    bool meets(const Span& o) const { return lo < o.hi && o.lo < hi; }
};

// Whether every output lies apart from every input and from every other output.
bool apart(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
    for (const Span* o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Span& i : inputs)
            if (o->meets(i)) return false;
        for (const Span* q = outputs.begin(); q != o; ++q)
            if (o->meets(*q)) return false;
    }
    return true;
}

bool valid_type(int t) { return t == MXG_F32 || t == MXG_BF16; }
bool valid_act(int a) { return a >= MXG_ACT_NONE && a <= MXG_ACT_SWIGLU; }

mxg_status check_norm_sizes(int64_t T, int64_t H) {
    if (H <= 0 || T < 0) return MXG_ERROR_INVALID_VALUE;
    if (H % 8 != 0 || H > INT32_MAX / 2 || T > INT32_MAX / 2) return MXG_ERROR_NOT_SUPPORTED;
    return MXG_SUCCESS;
}

mxg_status check_matmul_sizes(int64_t T, int64_t N, int64_t K, int32_t G, int32_t E, const void* off,
                              const void* ids) {
    if (K <= 0 || N <= 0 || E <= 0 || T < 0 || G < 0) return MXG_ERROR_INVALID_VALUE;
    if (K % 8 != 0 || K > MXG_MAX_K || N > INT32_MAX / 2 || T > INT32_MAX || G > MXG_MAX_GROUPS)
        return MXG_ERROR_NOT_SUPPORTED;
    if (G == 0) return MXG_SUCCESS;  // the routing is not looked at (an empty expert_ids has no address)
    if ((off == nullptr) != (ids == nullptr)) return MXG_ERROR_INVALID_VALUE;
    if (off == nullptr && (G != 1 || E != 1)) return MXG_ERROR_INVALID_VALUE;
    if (!aligned(off, 4) || !aligned(ids, 4)) return MXG_ERROR_INVALID_VALUE;
    return MXG_SUCCESS;
}

mxg_status check_groups(const uint32_t* off, const int32_t* ids, int32_t G, int32_t E, int64_t T, hipStream_t stream) {
    return off == nullptr ? MXG_SUCCESS : check_routing(off, ids, G, E, T, stream);
}

}  // namespace

extern "C" {

mxg_status mx_rmsnorm(mxg_norm_format format, mxg_dtype stream_type, const void* x, const void* residual,
                      mxg_dtype weight_type, const void* weight, float weight_offset, float eps, int64_t num_tokens,
                      int64_t H, void* h, void* y_bf16, void* q, void* scales, hipStream_t stream) {
    const int fmt = (int)format;
    if (fmt < MXG_NORM_PLAIN || fmt > MXG_NORM_FP8_BLOCK128 || !valid_type(stream_type) || !valid_type(weight_type) ||
        !(eps >= 0.0f))
        return MXG_ERROR_INVALID_VALUE;
    if (mxg_status st = check_norm_sizes(num_tokens, H)) return st;
    if (fmt != MXG_NORM_PLAIN && H % 32 != 0) return MXG_ERROR_NOT_SUPPORTED;
    if ((residual == nullptr) != (h == nullptr) || (q == nullptr) != (fmt == MXG_NORM_PLAIN) ||
        (scales == nullptr) != (fmt == MXG_NORM_PLAIN) || (!y_bf16 && !q)) {
        if (num_tokens > 0) return MXG_ERROR_INVALID_VALUE;
    }
    if (num_tokens == 0) return MXG_SUCCESS;  // nothing is read or written
    if (!x || !weight) return MXG_ERROR_INVALID_VALUE;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(h, 16) || !aligned(y_bf16, 16) ||
        !aligned(q, 16) || !aligned(scales, fmt == MXG_NORM_MXFP8 ? 1 : 4))
        return MXG_ERROR_INVALID_VALUE;
    const uint64_t T = (uint64_t)num_tokens, W = (uint64_t)H, size = stream_type == MXG_F32 ? 4 : 2;
    const uint64_t x_size = residual ? 2 : size;
    const Span xs(x, x_size, T, W), rs(residual, size, T, W), ws(weight, weight_type == MXG_F32 ? 4 : 2, W);
    const Span hs(h, size, T, W), none(nullptr, 1, 0);
    // h may take residual's place, or x's where both are bf16
    if (!apart({hs}, {h == x && x_size == size ? none : xs, h == residual ? none : rs, ws})) return MXG_ERROR_INVALID_VALUE;
    const Span ss = fmt == MXG_NORM_FP8_ROWWISE ? Span(scales, 4, T)
                    : fmt == MXG_NORM_MXFP8     ? Span(scales, 1, T, W / 32)
                                                : Span(scales, 4, T, (W + 127) / 128);
    if (!apart({Span(y_bf16, 2, T, W), Span(q, 1, T, W), ss}, {xs, rs, ws, hs})) return MXG_ERROR_INVALID_VALUE;
    return from_hip(mxg::launch_rmsnorm(fmt, stream_type == MXG_F32, x, residual, weight_type == MXG_F32, weight,
                                        weight_offset, eps, num_tokens, H, h, y_bf16, q, scales, stream));
}

int64_t mx_rmsnorm_workspace_bytes(int64_t num_tokens, int64_t H) {
    if (check_norm_sizes(num_tokens, H)) return -1;
    return mxg::rmsnorm_workspace_rows(num_tokens, H) * H * (int64_t)sizeof(float);
}

mxg_status mx_rmsnorm_backward(mxg_dtype stream_type, const void* dy_bf16, const void* h, mxg_dtype weight_type,
                               const void* weight, float weight_offset, float eps, const void* dh, int64_t num_tokens,
                               int64_t H, void* dx, void* dx_bf16, float* dweight, float* workspace,
                               hipStream_t stream) {
    if (!valid_type(stream_type) || !valid_type(weight_type) || !(eps >= 0.0f)) return MXG_ERROR_INVALID_VALUE;
    if (mxg_status st = check_norm_sizes(num_tokens, H)) return st;
    if (!dx && !dx_bf16 && !dweight) return MXG_ERROR_INVALID_VALUE;
    if (!aligned(dx, 16) || !aligned(dx_bf16, 16) || !aligned(dweight, 4)) return MXG_ERROR_INVALID_VALUE;
    if (num_tokens > 0) {
        if (!dy_bf16 || !h || !weight || (dweight && !workspace)) return MXG_ERROR_INVALID_VALUE;
        if (!aligned(dy_bf16, 16) || !aligned(h, 16) || !aligned(weight, 16) || !aligned(dh, 16) ||
            !aligned(workspace, 4))
            return MXG_ERROR_INVALID_VALUE;
        const uint64_t T = (uint64_t)num_tokens, W = (uint64_t)H, size = stream_type == MXG_F32 ? 4 : 2;
        const Span past(dx == dh ? nullptr : dh, size, T, W);  // dx may take dh's place
        if (!apart({Span(dx, size, T, W), Span(dx_bf16, 2, T, W), Span(dweight, 4, W),
                    Span(dweight ? workspace : nullptr, 4, (uint64_t)mxg::rmsnorm_workspace_rows(num_tokens, H), W)},
                   {Span(dy_bf16, 2, T, W), Span(h, size, T, W), Span(weight, weight_type == MXG_F32 ? 4 : 2, W), past}))
            return MXG_ERROR_INVALID_VALUE;
    } else if (!dweight) {
        return MXG_SUCCESS;  // nothing is read or written
    }
    return from_hip(mxg::launch_rmsnorm_backward(stream_type == MXG_F32, dy_bf16, h, weight_type == MXG_F32, weight,
                                                 weight_offset, eps, dh, num_tokens, H, dx, dx_bf16, dweight,
                                                 workspace, stream));
}

mxg_status mx_grouped_matmul_bf16(mxg_activation act, const void* a_bf16, const void* b_bf16, const float* bias,
                                  const void* residual, mxg_dtype c_type, void* c, void* z_bf16,
                                  const uint32_t* row_offsets, const int32_t* expert_ids, int32_t num_groups,
                                  int32_t num_experts, int64_t total_rows, int64_t N, int64_t K,
                                  int64_t max_rows_per_group_hint, hipStream_t stream) {
    if (!valid_act(act) || !valid_type(c_type)) return MXG_ERROR_INVALID_VALUE;
    if (mxg_status st = check_matmul_sizes(total_rows, N, K, num_groups, num_experts, row_offsets, expert_ids))
        return st;
    if (act == MXG_ACT_SWIGLU && N % 2 != 0) return MXG_ERROR_NOT_SUPPORTED;
    if (total_rows == 0 || num_groups == 0) return MXG_SUCCESS;  // nothing is read or written
    if (!a_bf16 || !b_bf16 || !c) return MXG_ERROR_INVALID_VALUE;
    if (!aligned(a_bf16, 16) || !aligned(b_bf16, 16) || !aligned(bias, 4) || !aligned(residual, 16) ||
        !aligned(c, 16) || !aligned(z_bf16, 16))
        return MXG_ERROR_INVALID_VALUE;
    const uint64_t T = (uint64_t)total_rows, E = (uint64_t)num_experts, W = (uint64_t)N, D = (uint64_t)K;
    const uint64_t wide = act == MXG_ACT_SWIGLU ? W / 2 : W, size = c_type == MXG_F32 ? 4 : 2;
    // c may take residual's place
    if (!apart({Span(c, size, T, wide), Span(z_bf16, 2, T, W)},
               {Span(a_bf16, 2, T, D), Span(b_bf16, 2, E, W, D), Span(bias, 4, E, W),
                Span(residual == c ? nullptr : residual, size, T, wide)}))
        return MXG_ERROR_INVALID_VALUE;
    if (mxg_status st = check_groups(row_offsets, expert_ids, num_groups, num_experts, total_rows, stream)) return st;
    const mxg::Bf16Problem p{(int)act, a_bf16, b_bf16, bias, residual, c, c_type == MXG_F32, z_bf16, row_offsets,
                             expert_ids, num_groups, num_experts, total_rows, N, K, max_rows_per_group_hint,
                             aligned(bias, 16)};
    return from_hip(mxg::launch_matmul_bf16(p, stream));
}

mxg_status mx_grouped_matmul_bf16_backward(mxg_activation act, const void* dc_bf16, const void* b_bf16,
                                           const void* z_bf16, void* da_bf16, const uint32_t* row_offsets,
                                           const int32_t* expert_ids, int32_t num_groups, int32_t num_experts,
                                           int64_t total_rows, int64_t N, int64_t K, int64_t max_rows_per_group_hint,
                                           hipStream_t stream) {
    if (!valid_act(act)) return MXG_ERROR_INVALID_VALUE;
    if (mxg_status st = check_matmul_sizes(total_rows, N, K, num_groups, num_experts, row_offsets, expert_ids))
        return st;
    if (N % 8 != 0 || N > MXG_MAX_K) return MXG_ERROR_NOT_SUPPORTED;
    if (total_rows == 0 || num_groups == 0) return MXG_SUCCESS;  // nothing is read or written
    if (!dc_bf16 || !b_bf16 || !da_bf16 || (z_bf16 == nullptr) != (act == MXG_ACT_NONE))
        return MXG_ERROR_INVALID_VALUE;
    if (!aligned(dc_bf16, 16) || !aligned(b_bf16, 16) || !aligned(z_bf16, 16) || !aligned(da_bf16, 16))
        return MXG_ERROR_INVALID_VALUE;
    const uint64_t T = (uint64_t)total_rows, wide = (uint64_t)K * (act == MXG_ACT_SWIGLU ? 2 : 1);
    // da may take z's place
    if (!apart({Span(da_bf16, 2, T, wide)},
               {Span(dc_bf16, 2, T, (uint64_t)N), Span(b_bf16, 2, (uint64_t)num_experts, (uint64_t)N, (uint64_t)K),
                Span(z_bf16 == da_bf16 ? nullptr : z_bf16, 2, T, wide)}))
        return MXG_ERROR_INVALID_VALUE;
    if (mxg_status st = check_groups(row_offsets, expert_ids, num_groups, num_experts, total_rows, stream)) return st;
    const mxg::Bf16Problem p{(int)act, dc_bf16, b_bf16, nullptr, nullptr, da_bf16, false, const_cast<void*>(z_bf16),
                             row_offsets, expert_ids, num_groups, num_experts, total_rows, N, K,
                             max_rows_per_group_hint, false};
    return from_hip(mxg::launch_matmul_bf16_backward(p, stream));
}

mxg_status mx_grouped_matmul_bf16_backward_weights(const void* dc_bf16, const void* a_bf16, mxg_dtype dw_type,
                                                   void* dw, float* dbias, int32_t accumulate,
                                                   const uint32_t* row_offsets, const int32_t* expert_ids,
                                                   int32_t num_groups, int32_t num_experts, int64_t total_rows,
                                                   int64_t N, int64_t K, hipStream_t stream) {
    if (!valid_type(dw_type)) return MXG_ERROR_INVALID_VALUE;
    if (mxg_status st = check_matmul_sizes(total_rows, N, K, num_groups, num_experts, row_offsets, expert_ids))
        return st;
    if (N % 8 != 0 || N > MXG_MAX_K) return MXG_ERROR_NOT_SUPPORTED;
    if (!dw || !aligned(dw, 16) || !aligned(dbias, 4)) return MXG_ERROR_INVALID_VALUE;
    if (total_rows > 0 && num_groups > 0) {
        if (!dc_bf16 || !a_bf16 || !aligned(dc_bf16, 16) || !aligned(a_bf16, 16)) return MXG_ERROR_INVALID_VALUE;
        const uint64_t T = (uint64_t)total_rows, E = (uint64_t)num_experts, W = (uint64_t)N, D = (uint64_t)K;
        if (!apart({Span(dw, dw_type == MXG_F32 ? 4 : 2, E, W, D), Span(dbias, 4, E, W)},
                   {Span(dc_bf16, 2, T, W), Span(a_bf16, 2, T, D)}))
            return MXG_ERROR_INVALID_VALUE;
        if (mxg_status st = check_groups(row_offsets, expert_ids, num_groups, num_experts, total_rows, stream))
            return st;
    } else if (accumulate != 0) {
        return MXG_SUCCESS;  // nothing to add
    } else {
        num_groups = 0;  // zeros, without a look at the routing
    }
    return from_hip(mxg::launch_matmul_bf16_weights(dc_bf16, a_bf16, dw, dw_type == MXG_F32, dbias, accumulate != 0,
                                                    row_offsets, expert_ids, num_groups, num_experts, total_rows, N,
                                                    K, stream));
}

mxg_status mx_activation_backward(mxg_activation act, const void* dc_bf16, const void* z_bf16, void* dz_bf16,
                                  int64_t num_rows, int64_t N, hipStream_t stream) {
    if (!valid_act(act) || N <= 0 || num_rows < 0) return MXG_ERROR_INVALID_VALUE;
    if (N % 8 != 0 || N > INT32_MAX / 2 || num_rows > INT32_MAX) return MXG_ERROR_NOT_SUPPORTED;
    if (num_rows == 0) return MXG_SUCCESS;  // nothing is read or written
    if (act == MXG_ACT_NONE || !dc_bf16 || !z_bf16 || !dz_bf16) return MXG_ERROR_INVALID_VALUE;
    if (!aligned(dc_bf16, 16) || !aligned(z_bf16, 16) || !aligned(dz_bf16, 16)) return MXG_ERROR_INVALID_VALUE;
    const uint64_t T = (uint64_t)num_rows, W = (uint64_t)N, wide = act == MXG_ACT_SWIGLU ? 2 * W : W;
    const void* dc_apart = dz_bf16 == dc_bf16 && wide == W ? nullptr : dc_bf16;  // dz may take z's or dc's place
    if (!apart({Span(dz_bf16, 2, T, wide)}, {Span(dz_bf16 == z_bf16 ? nullptr : z_bf16, 2, T, wide), Span(dc_apart, 2, T, W)}))
        return MXG_ERROR_INVALID_VALUE;
    return from_hip(mxg::launch_activation_backward((int)act, dc_bf16, z_bf16, dz_bf16, num_rows, N, stream));
}

int32_t mxg_bf16_tile(mxg_bf16_product product, int32_t num_groups, int32_t num_experts, int64_t total_rows, int64_t N,
                      int64_t K, int64_t max_rows_per_group_hint) {
    if (num_groups <= 0 || total_rows <= 0 || check_matmul_sizes(total_rows, N, K, num_groups, num_experts, &N, &N))
        return 0;
    if (product != MXG_BF16_FORWARD && (N % 8 != 0 || N > MXG_MAX_K)) return 0;
    if (product == MXG_BF16_BACKWARD_WEIGHTS)
        return mxg::bf16_weights_tile_choice(num_groups, num_experts, total_rows, N, K);
    if (product != MXG_BF16_FORWARD && product != MXG_BF16_BACKWARD) return 0;
    mxg::Bf16Problem p{};
    p.G = num_groups;
    p.E = num_experts;
    p.T = total_rows;
    p.N = N;
    p.K = K;
    p.max_rows_hint = max_rows_per_group_hint;
    return mxg::bf16_tile_choice(p, product == MXG_BF16_BACKWARD);
}

}  // extern "C"
