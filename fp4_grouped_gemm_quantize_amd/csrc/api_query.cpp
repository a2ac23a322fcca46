// api_query.cpp -- the extern "C" question which kernel a block-128 grouped GEMM
// of given sizes runs.  Host code only; nothing is enqueued.
#include "api_common.h"

extern "C" {

int32_t mxg_block128_tile(int32_t num_groups, int64_t total_rows, int64_t N, int64_t K,
                          int64_t max_rows_per_group_hint) {
    if (num_groups <= 0 || total_rows <= 0 || N <= 0 || K <= 0) return 0;
    if (K % 32 != 0 || K > MXG_MAX_K || num_groups > MXG_MAX_GROUPS || N > INT32_MAX / 2 || total_rows > INT32_MAX)
        return 0;
    mxg::GemmProblem p{};
    p.G = num_groups;
    p.T = total_rows;
    p.N = N;
    p.K = K;
    p.max_rows_hint = max_rows_per_group_hint;
    return mxg::block128_tile_choice(p);
}

}  // extern "C"
