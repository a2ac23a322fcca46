// Drives api_dense.cpp (linked with the host-only stand-ins below) through its
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
hipError_t launch_rmsnorm(int, bool, const void*, const void*, bool, const void*, float, float, int64_t, int64_t, void*,
                          void*, void*, void*, hipStream_t) {
    return record("rmsnorm");
}
int64_t rmsnorm_workspace_rows(int64_t T, int64_t) { return T < 512 ? T : 512; }
hipError_t launch_rmsnorm_backward(bool, const void*, const void*, bool, const void*, float, float, const void*,
                                   int64_t, int64_t, void*, void*, float*, float*, hipStream_t) {
    return record("rmsnorm_backward");
}
hipError_t launch_matmul_bf16(const Bf16Problem&, hipStream_t) { return record("matmul"); }
hipError_t launch_matmul_bf16_backward(const Bf16Problem&, hipStream_t) { return record("backward"); }
hipError_t launch_matmul_bf16_weights(const void*, const void*, void*, bool, float*, bool, const uint32_t*,
                                      const int32_t*, int, int, int64_t, int64_t, int64_t, hipStream_t) {
    return hipErrorInvalidValue;
}
hipError_t launch_activation_backward(int, const void*, const void*, void*, int64_t, int64_t, hipStream_t) {
    return record("activation");
}
int bf16_tile_choice(const Bf16Problem&, bool back) { return back ? 2 : 1; }
int bf16_weights_tile_choice(int, int, int64_t, int64_t, int64_t) { return 3; }
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
    alignas(16) static unsigned char buf[8][4096];
    const uint32_t off[3] = {0, 2, 4}, bad[3] = {0, 3, 2};
    const int32_t ids[2] = {1, 0}, far_ids[2] = {1, 9};
    for (int validate = 0; validate < 2; ++validate) {
        if (validate) setenv("MXG_VALIDATE", "1", 1);
        else unsetenv("MXG_VALIDATE");
        const mxg_status refused = validate ? MXG_ERROR_INVALID_VALUE : MXG_SUCCESS;
        const int kept = validate ? 0 : 1;
        expect(mx_rmsnorm(MXG_NORM_FP8_BLOCK128, MXG_BF16, buf[0], buf[1], MXG_F32, buf[2], 0.f, 1e-6f, 4, 64, buf[1],
                          buf[3], buf[4], buf[5], nullptr),
               MXG_SUCCESS, 1, "norm, h in the residual's place");
        expect(mx_rmsnorm(MXG_NORM_PLAIN, MXG_BF16, buf[0], buf[1], MXG_BF16, buf[2], 0.f, 0.f, 4, 64, buf[0], buf[3],
                          nullptr, nullptr, nullptr),
               MXG_SUCCESS, 1, "norm, h in x's place");
        expect(mx_rmsnorm(MXG_NORM_PLAIN, MXG_F32, buf[0], buf[1], MXG_BF16, buf[2], 0.f, 0.f, 4, 64, buf[0], buf[3],
                          nullptr, nullptr, nullptr),
               MXG_ERROR_INVALID_VALUE, 0, "norm, an fp32 h over a bf16 x");
        expect(mx_rmsnorm_backward(MXG_F32, buf[0], buf[1], MXG_BF16, buf[2], 1.f, 1e-6f, buf[3], 4, 64, buf[3], buf[4],
                                   (float*)buf[5], (float*)buf[6], nullptr),
               MXG_SUCCESS, 1, "norm's gradient, dx in dh's place");
        expect(mx_rmsnorm_backward(MXG_F32, nullptr, nullptr, MXG_BF16, nullptr, 1.f, 1e-6f, nullptr, 0, 64, nullptr,
                                   nullptr, (float*)buf[5], nullptr, nullptr),
               MXG_SUCCESS, 1, "norm's gradient of no tokens");
        for (const void* residual : {(const void*)buf[3], (const void*)buf[2], (const void*)nullptr})
            expect(mx_grouped_matmul_bf16(MXG_ACT_SILU, buf[0], buf[1], (float*)buf[4], residual, MXG_BF16, buf[2],
                                          buf[5], off, ids, 2, 2, 4, 16, 32, 0, nullptr),
                   MXG_SUCCESS, 1, "product");
        expect(mx_grouped_matmul_bf16(MXG_ACT_NONE, buf[0], buf[1], nullptr, nullptr, MXG_F32, buf[2], nullptr, bad, ids,
                                      2, 2, 4, 16, 32, 0, nullptr),
               refused, kept, "product, bad offsets");
        expect(mx_grouped_matmul_bf16(MXG_ACT_NONE, buf[0], buf[1], nullptr, nullptr, MXG_F32, buf[2], nullptr, nullptr,
                                      nullptr, 1, 1, 4, 16, 32, 0, nullptr),
               MXG_SUCCESS, 1, "dense product");
        expect(mx_grouped_matmul_bf16_backward(MXG_ACT_SWIGLU, buf[0], buf[1], buf[2], buf[2], off, ids, 2, 2, 4, 16, 32,
                                               0, nullptr),
               MXG_SUCCESS, 1, "rows' gradient in z's place");
        expect(mx_grouped_matmul_bf16_backward(MXG_ACT_NONE, buf[0], buf[1], nullptr, buf[2], off, far_ids, 2, 2, 4, 16,
                                               32, 0, nullptr),
               refused, kept, "rows' gradient, bad ids");
        expect(mx_activation_backward(MXG_ACT_RELU, buf[0], buf[1], buf[0], 4, 16, nullptr), MXG_SUCCESS, 1,
               "activation in dc's place");
        // the stand-in refuses the launch: reported as such
        expect(mx_grouped_matmul_bf16_backward_weights(buf[0], buf[1], MXG_F32, buf[2], (float*)buf[3], 0, off, ids, 2, 2,
                                                       4, 16, 32, nullptr),
               MXG_ERROR_LAUNCH, 0, "weights' gradient");
        expect(mx_grouped_matmul_bf16_backward_weights(nullptr, nullptr, MXG_F32, buf[2], nullptr, 0, nullptr, nullptr, 0,
                                                       2, 0, 16, 32, nullptr),
               MXG_ERROR_LAUNCH, 0, "zeros where there are no rows");
        expect(mx_grouped_matmul_bf16_backward_weights(nullptr, nullptr, MXG_F32, buf[2], nullptr, 1, nullptr, nullptr, 0,
                                                       2, 0, 16, 32, nullptr),
               MXG_SUCCESS, 0, "nothing to add");
        if (mxg_bf16_tile(MXG_BF16_BACKWARD, 1, 1, 4, 16, 32, 0) != 2 ||
            mxg_bf16_tile(MXG_BF16_BACKWARD_WEIGHTS, 1, 1, 4, 16, 32, 0) != 3 ||
            mxg_bf16_tile(MXG_BF16_FORWARD, 1, 1, 4, 15, 32, 0) != 1)
            ++g_fails;
    }
    printf("fails %d\n", g_fails);
    return g_fails != 0;
}
