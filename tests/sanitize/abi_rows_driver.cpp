// Drives the MXG_VALIDATE check of the block-128 scatter's row_of_slot in
// api_moe.cpp, with the host-only stand-ins of abi_moe_driver.cpp; "device"
// pointers are host memory here.  Prints "fails N".
#define main moe_driver_main
#include "abi_moe_driver.cpp"
#undef main

int main() {
    alignas(16) static unsigned char buf[4096];
    float f[16] = {};
    const uint32_t off[3] = {1, 2, 4}, none[3] = {2, 2, 2};  // rows 1, 2 and 3 covered; no row covered
    const int32_t once[4] = {3, 1, -1, 2};
    const int32_t twice[4] = {3, 1, 2, 3}, edges[4] = {1, 2, 5, 1};
    const int32_t outside[4] = {0, 2, 0, 0};    // row 0 lies in no group: dropped as often as named
    const int32_t behind[4] = {4, 4, 7, 7};     // past the groups, past the rows
    const int32_t strange[4] = {INT32_MIN, INT32_MAX, INT32_MIN, INT32_MAX};
    auto scatter = [&](const int32_t* ros, const uint32_t* o, int64_t T) {
        return mx_grouped_quantize_block128_scatter(buf, 2, ros, 2, buf, f, o, 2, T, 32, nullptr);
    };
    for (int validate = 0; validate < 2; ++validate) {
        if (validate) setenv("MXG_VALIDATE", "1", 1);
        else unsetenv("MXG_VALIDATE");
        const mxg_status refused = validate ? MXG_ERROR_INVALID_VALUE : MXG_SUCCESS;
        const int kept = validate ? 0 : 1;
        expect(scatter(once, off, 5), MXG_SUCCESS, 1, "rows named once");
        expect(scatter(twice, off, 5), refused, kept, "a covered row named twice");
        expect(scatter(edges, off, 5), refused, kept, "the first covered row named twice");
        expect(scatter(outside, off, 5), MXG_SUCCESS, 1, "an uncovered row named twice");
        expect(scatter(behind, off, 5), MXG_SUCCESS, 1, "rows behind the groups and past the end named twice");
        expect(scatter(strange, off, INT32_MAX), MXG_SUCCESS, 1, "indices at the ends of their type");
        expect(scatter(twice, none, 5), MXG_SUCCESS, 1, "no row covered");
    }
    printf("fails %d\n", g_fails);
    return g_fails != 0;
}
