// Drives api_moe.cpp (linked with the host-only stand-ins below) through its
// launches and through the MXG_VALIDATE checks; "device" pointers are host
// memory here.  Prints "fails N".
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "mxg.h"
#include "mxg_internal.h"

static int g_launches = 0, g_fails = 0;
static const char* g_last = "";
static hipError_t record(const char* what) {
    ++g_launches;
    g_last = what;
    return hipSuccess;
}

namespace mxg {
hipError_t launch_topk(int, int, const void*, const float*, int64_t, int, int, bool, float, int32_t*, float*,
                       hipStream_t) {
    return record("topk");
}
hipError_t launch_topk_backward(int, int, const void*, const int32_t*, const float*, int64_t, int, int, bool, float,
                                void*, hipStream_t) {
    return record("topk_backward");
}
hipError_t launch_sort(const int32_t*, int64_t, int, uint32_t*, int32_t*, int32_t*, hipStream_t) {
    return record("sort");
}
hipError_t launch_permute(const void*, int64_t, int64_t, const int32_t*, int, void*, int64_t, hipStream_t) {
    return record("permute");
}
hipError_t launch_permute_backward(const void*, int64_t, int64_t, const int32_t*, int64_t, int, void*, hipStream_t) {
    return record("permute_backward");
}
hipError_t launch_combine_backward(const void*, const void*, int64_t, int64_t, const int32_t*, const float*, int64_t,
                                   int, void*, float*, hipStream_t) {
    return record("combine_backward");
}
hipError_t launch_quantize_block128(const void*, int64_t, const int32_t*, int, void*, float*, const uint32_t*, int,
                                    int64_t, int64_t, hipStream_t) {
    return record("quantize_block128");
}
hipError_t launch_quantize_weights_block128(const void*, int64_t, int64_t, int64_t, void*, float*, void*, float*,
                                            hipStream_t) {
    return record("quantize_weights_block128");
}
hipError_t launch_silu_quantize_block128(const void*, void*, float*, const uint32_t*, int, int64_t, int64_t,
                                         hipStream_t) {
    return record("silu_quantize_block128");
}
hipError_t launch_silu_backward_block128(const void*, const void*, void*, void*, float*, const uint32_t*, int, int64_t,
                                         int64_t, hipStream_t) {
    return record("silu_backward_block128");
}
hipError_t launch_grouped_gemm_block128(const GemmProblem&, hipStream_t) { return hipErrorInvalidValue; }
}  // namespace mxg

extern "C" {
hipError_t hipMemcpyAsync(void* dst, const void* src, size_t n, hipMemcpyKind, hipStream_t) {
    memcpy(dst, src, n);
    return hipSuccess;
}
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
}

static void expect(mxg_status got, mxg_status want, int launches, const char* what) {
    if (got != want || g_launches != launches) {
        printf("FAIL %s: status %d (want %d), launches %d (want %d), last %s\n", what, (int)got, (int)want, g_launches,
               launches, g_last);
        ++g_fails;
    }
    g_launches = 0;
}

int main() {
    alignas(16) static unsigned char buf[4096];
    const int32_t rows[4] = {2, 0, -1, 1}, twice[4] = {2, 0, 7, 2};
    const uint32_t off[3] = {0, 2, 4}, bad[3] = {0, 3, 2};
    const int32_t ids[2] = {1, 0}, far_ids[2] = {1, 9};
    float f[16] = {};
    for (int validate = 0; validate < 2; ++validate) {
        if (validate) setenv("MXG_VALIDATE", "1", 1);
        else unsetenv("MXG_VALIDATE");
        const mxg_status refused = validate ? MXG_ERROR_INVALID_VALUE : MXG_SUCCESS;
        const int kept = validate ? 0 : 1;
        expect(mx_moe_topk(MXG_F32, MXG_SCORE_SOFTMAX, buf, nullptr, 2, 4, 2, 1, 1.f, (int32_t*)buf, f, nullptr),
               MXG_SUCCESS, 1, "topk");
        expect(mx_moe_topk_backward(MXG_BF16, MXG_SCORE_SIGMOID, buf + 2, rows, f, 2, 4, 2, 0, 1.f, buf + 2, nullptr),
               MXG_SUCCESS, 1, "topk_backward");
        expect(mx_moe_sort(rows, 2, 2, 3, (uint32_t*)buf, (int32_t*)buf, (int32_t*)buf, nullptr), MXG_SUCCESS, 1,
               "sort");
        expect(mx_moe_sort(nullptr, 0, 2, 3, (uint32_t*)buf, nullptr, nullptr, nullptr), MXG_SUCCESS, 1, "sort of none");
        expect(mx_moe_permute(buf, 2, 8, rows, 2, buf, 4, nullptr), MXG_SUCCESS, 1, "permute");
        expect(mx_moe_permute(buf, 2, 8, twice, 2, buf, 4, nullptr), refused, kept, "permute of repeated rows");
        expect(mx_moe_permute_backward(buf, 4, 8, twice, 2, 2, buf, nullptr), MXG_SUCCESS, 1, "permute_backward");
        expect(mx_moe_combine_backward(buf, buf, 4, 8, rows, f, 2, 2, buf, f, nullptr), MXG_SUCCESS, 1,
               "combine_backward");
        expect(mx_moe_combine_backward(buf, buf, 4, 8, twice, f, 2, 2, buf, f, nullptr), refused, kept,
               "combine_backward of repeated rows");
        // more rows than an int32 can name, more than there is memory for: no exception leaves
        expect(mx_moe_permute(buf, 2, 8, rows, 2, buf, INT64_MAX, nullptr), MXG_SUCCESS, 1, "permute into many rows");
        expect(mx_moe_combine_backward(buf, buf, INT64_MAX, 8, twice, f, 2, 2, buf, f, nullptr), refused, kept,
               "combine_backward of many rows, repeated");
        expect(mx_moe_combine_backward(buf, nullptr, 0, 8, rows, f, 2, 2, nullptr, f, nullptr), MXG_SUCCESS, 1,
               "combine_backward without rows");
        expect(mx_grouped_quantize_block128(buf, buf, f, off, 2, 4, 32, nullptr), MXG_SUCCESS, 1, "quantize");
        expect(mx_grouped_quantize_block128(buf, buf, f, bad, 2, 4, 32, nullptr), refused, kept, "quantize, bad offsets");
        expect(mx_grouped_quantize_block128_scatter(buf, 2, rows, 2, buf, f, off, 2, 4, 32, nullptr), MXG_SUCCESS, 1,
               "scatter");
        expect(mx_quantize_weights_block128(buf, 1, 32, 32, buf, f, nullptr, nullptr, nullptr), MXG_SUCCESS, 1,
               "weights");
        expect(mx_silu_quantize_block128(buf, buf, f, off, 2, 4, 32, nullptr), MXG_SUCCESS, 1, "silu");
        expect(mx_silu_backward_block128(buf, buf, buf, nullptr, nullptr, off, 2, 4, 32, nullptr), MXG_SUCCESS, 1,
               "silu_backward");
        expect(mx_silu_backward_block128(buf, buf, buf, nullptr, nullptr, bad, 2, 4, 32, nullptr), refused, kept,
               "silu_backward, bad offsets");
        // the stand-in refuses the launch: reported as such
        expect(mx_grouped_matmul_block128(buf, f, buf, f, buf, off, ids, 2, 2, 4, 8, 32, 0, nullptr), MXG_ERROR_LAUNCH,
               0, "gemm");
        expect(mx_grouped_matmul_block128(buf, f, buf, f, buf, off, far_ids, 2, 2, 4, 8, 32, 0, nullptr),
               validate ? MXG_ERROR_INVALID_VALUE : MXG_ERROR_LAUNCH, 0, "gemm, bad ids");
    }
    printf("fails %d\n", g_fails);
    return g_fails != 0;
}
