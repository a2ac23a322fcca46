// fp8_encode.h -- what the kernels that encode FP8 e4m3 under an fp32 scale share:
// block maxima that keep NaN, the codes of 8 values under their scale, and an
// 8-byte nontemporal store.  Device code for gfx950.
#pragma once

#include "mxg_device.h"

namespace mxg {

// Largest magnitude of 8 values, as the integer order of the magnitudes has it:
// a NaN's pattern lies above infinity's, so a block with a NaN gets a NaN scale
// (a floating-point maximum would drop it).
__device__ __forceinline__ float amax8(const float* f) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(f[i]) & 0x7fffffffu);
    return __uint_as_float(a);
}
// The same maximum over 8 (16) neighbouring lanes: lane ^ 1, lane ^ 2, then the
// mirrors within 8 (and 16) lanes.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float amax_of8(float v) {
    return __uint_as_float(dpp_umax<0x141>(dpp_umax<0x4E>(dpp_umax<0xB1>(__float_as_uint(v)))));
}
__device__ __forceinline__ float amax_of16(float v) {
    return __uint_as_float(dpp_umax<0x140>(__float_as_uint(amax_of8(v))));
}

// Codes of 8 values under their block's scale: e4m3(x / scale), the code of the
// quotient that IEEE binary32 division gives.  One division gives the scale's
// reciprocal r; each quotient is then x r corrected by its exact remainder,
// q + (x - q scale) r (Markstein), three operations instead of a division's ten.
// Scales below 2^-60 are lifted by 2^64 with their values, an exact step, so that
// neither the reciprocal overflows nor the remainder underflows.  (Checked on the
// CPU: the codes equal those of the division for every bf16 maximum and every bf16
// value up to it, and for 480 M fp32 pairs, half of them next to a code's border;
// only quotients far below the smallest code differ from the division's.)  Under an
// infinite scale r is 0 and the remainder is taken with the largest finite number
// instead, since 0 times infinity would make the quotient of a finite value, 0, a
// NaN; an infinity over it stays one.  The clamp matters only where the scale is a
// subnormal that rounded down.
__device__ __forceinline__ uint2 encode8(const float* x, float scale) {
    float f[8];
    if (scale == 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = x[i] * 0.0f;
    } else {
        const float lift = scale < 0x1p-60f ? 0x1p64f : 1.0f;
        const float lifted = scale * lift, r = 1.0f / lifted, s = fminf(lifted, 0x1.fffffep127f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float xi = x[i] * lift, q = xi * r;
            const float v = copysignf(fmaf(fmaf(-q, s, xi), r, q), q);  // (a remainder of 0 would turn -0 into 0)
            f[i] = v > 448.0f ? 448.0f : v < -448.0f ? -448.0f : v;  // keeps a NaN
        }
    }
    return pack8_e4m3(f);
}

// 8 bytes with the nontemporal hint.
__device__ __forceinline__ void store_stream8(void* p, const uint2& v) {
    typedef unsigned u2v __attribute__((ext_vector_type(2)));
    u2v t;
    t.x = v.x;
    t.y = v.y;
    __builtin_nontemporal_store(t, static_cast<u2v*>(p));
}

}  // namespace mxg
