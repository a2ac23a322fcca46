// api_common.h -- what the extern "C" layer's files share: pointer checks, the
// status of a launch, and the MXG_VALIDATE check of the routing metadata.  Host
// code only.
#pragma once

#include "mxg.h"
#include "mxg_internal.h"

#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <exception>
#include <vector>

namespace mxg {
namespace api {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline mxg_status from_hip(hipError_t e) { return e == hipSuccess ? MXG_SUCCESS : MXG_ERROR_LAUNCH; }

inline bool valid_fmt(int fmt) { return fmt == MXG_FP8_E4M3_ROWWISE || fmt == MXG_MXFP8_E4M3 || fmt == MXG_MXFP4_E2M1; }

// ---- MXG_VALIDATE: the optional check of the routing metadata (a debug mode).
inline thread_local char t_validation_msg[192] = "";

inline bool validation_on() {
    const char* v = getenv("MXG_VALIDATE");
    return v != nullptr && v[0] != '\0' && strcmp(v, "0") != 0;
}

// First violation in host copies of row_offsets [G + 1] and (if E > 0)
// expert_ids [G], written to `msg`; false if the routing is well formed.
inline bool find_violation(const uint32_t* off, const int32_t* ids, int64_t G, int64_t E, int64_t T, char* msg,
                    size_t len) {
    for (int64_t g = 0; g <= G; ++g) {
        if ((int64_t)off[g] > T) {
            snprintf(msg, len, "row_offsets[%lld] = %u exceeds total_rows = %lld", (long long)g, off[g],
                     (long long)T);
            return true;
        }
        if (g > 0 && off[g] < off[g - 1]) {
            snprintf(msg, len, "row_offsets[%lld] = %u is below row_offsets[%lld] = %u", (long long)g, off[g],
                     (long long)(g - 1), off[g - 1]);
            return true;
        }
    }
    if (ids != nullptr && E > 0)
        for (int64_t g = 0; g < G; ++g)
            if (ids[g] < 0 || ids[g] >= E) {
                snprintf(msg, len, "expert_ids[%lld] = %d lies outside [0, %lld)", (long long)g, ids[g],
                         (long long)E);
                return true;
            }
    return false;
}

// With MXG_VALIDATE set: copy the routing metadata to the host (synchronising
// `stream`) and refuse malformed routing before anything is launched.
// ids / E: the expert ids are checked when the entry point takes num_experts.
inline mxg_status check_routing(const uint32_t* off, const int32_t* ids, int64_t G, int64_t E, int64_t T,
                         hipStream_t stream) {
    if (!validation_on()) return MXG_SUCCESS;
    t_validation_msg[0] = '\0';
    try {
        std::vector<uint32_t> h_off((size_t)G + 1);
        std::vector<int32_t> h_ids(ids != nullptr && E > 0 ? (size_t)G : 0);
        if (hipMemcpyAsync(h_off.data(), off, sizeof(uint32_t) * h_off.size(), hipMemcpyDeviceToHost, stream) !=
            hipSuccess)
            return MXG_ERROR_LAUNCH;
        if (!h_ids.empty() && hipMemcpyAsync(h_ids.data(), ids, sizeof(int32_t) * h_ids.size(), hipMemcpyDeviceToHost,
                                             stream) != hipSuccess)
            return MXG_ERROR_LAUNCH;
        if (hipStreamSynchronize(stream) != hipSuccess) return MXG_ERROR_LAUNCH;
        if (find_violation(h_off.data(), h_ids.empty() ? nullptr : h_ids.data(), G, E, T, t_validation_msg,
                           sizeof t_validation_msg))
            return MXG_ERROR_INVALID_VALUE;
    } catch (const std::exception&) {
        return MXG_ERROR_LAUNCH;  // no exception leaves an entry point
    }
    return MXG_SUCCESS;
}

}  // namespace api
}  // namespace mxg
