// Host-only stand-ins for the HIP calls that libmxg's launchers make, as a library that is loaded before
// it: each launch is recorded instead of made, so that its size can be looked at where there is no GPU
// and no tensor behind the pointers.
#include <hip/hip_runtime_api.h>

#include <stdint.h>

static dim3 g_grid, g_block;
static uint64_t g_launches = 0, g_most_threads = 0;

extern "C" {

void recorder_reset() { g_launches = g_most_threads = 0; }
uint64_t recorder_launches() { return g_launches; }
uint64_t recorder_most_threads() { return g_most_threads; }  // of a launch

hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t) {
    g_grid = grid;
    g_block = block;
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream) {
    *grid = g_grid;
    *block = g_block;
    *shared = 0;
    *stream = nullptr;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3 grid, dim3 block, void**, size_t, hipStream_t) {
    const uint64_t workgroups = (uint64_t)grid.x * grid.y * grid.z, threads = (uint64_t)block.x * block.y * block.z;
    ++g_launches;
    if (workgroups * threads > g_most_threads) g_most_threads = workgroups * threads;
    return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipGetDevice(int* device) {
    *device = 0;
    return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* value, hipDeviceAttribute_t, int) {
    *value = 256;  // compute units
    return hipSuccess;
}
hipError_t hipOccupancyMaxActiveBlocksPerMultiprocessor(int* blocks, const void*, int, size_t) {
    *blocks = 8;
    return hipSuccess;
}

}  // extern "C"
