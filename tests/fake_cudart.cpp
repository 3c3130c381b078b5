// A CUDA runtime without a GPU, for host tests of the library's launches: the
// library's own objects linked with this file instead of cudart.  Kernels are
// not run; what a launch needs from the runtime is kept per device, as the
// runtime keeps it: a kernel's limit of dynamic shared memory is 48 KB until
// cudaFuncSetAttribute raises it for the current device, and a launch above
// the limit fails.
#include <cuda.h>
#include <cuda_runtime_api.h>

#include <atomic>
#include <chrono>
#include <cstring>
#include <map>
#include <mutex>
#include <thread>
#include <utility>

namespace {
int g_device = 0;
int g_launches = 0;
std::map<std::pair<const void *, int>, size_t> g_limit;  // (kernel, device) -> bytes
std::mutex g_mutex;
thread_local struct {
    dim3 grid, block;
    size_t smem;
    cudaStream_t stream;
} g_config;
char g_area[256];
std::atomic<int> g_lookups{0}, g_failing_lookups{0};

cudaError_t launch(const void *func, size_t smem) {
    std::lock_guard<std::mutex> lock(g_mutex);
    const auto it = g_limit.find({func, g_device});
    if (smem > (it == g_limit.end() ? 48u * 1024u : it->second)) return cudaErrorInvalidValue;
    ++g_launches;
    return cudaSuccess;
}

CUresult encode_tiled(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                      const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                      CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    return CUDA_SUCCESS;
}
}  // namespace

#define API extern "C" __attribute__((visibility("default")))

API void fake_set_device(int dev) { g_device = dev; }
API int fake_launches() { return g_launches; }
API int fake_lookups() { return g_lookups; }                        // of driver entry points
API void fake_fail_lookups(int n) { g_failing_lookups = n; }  // the next n find nothing

API cudaError_t cudaGetDevice(int *dev) {
    *dev = g_device;
    return cudaSuccess;
}
API cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr attr, int) {
    *v = attr == cudaDevAttrComputeCapabilityMajor ? 10 : attr == cudaDevAttrMultiProcessorCount ? 148 : 0;
    return cudaSuccess;
}
API cudaError_t cudaFuncSetAttribute(const void *func, cudaFuncAttribute attr, int value) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (attr == cudaFuncAttributeMaxDynamicSharedMemorySize) g_limit[{func, g_device}] = (size_t)value;
    return cudaSuccess;
}
API cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *cfg, const void *func, void **) {
    return launch(func, cfg->dynamicSmemBytes);
}
API cudaError_t cudaLaunchKernel(const void *func, dim3, dim3, void **, size_t smem, cudaStream_t) {
    return launch(func, smem);
}
API unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, cudaStream_t stream) {
    g_config = {grid, block, smem, stream};
    return 0;
}
API cudaError_t __cudaPopCallConfiguration(dim3 *grid, dim3 *block, size_t *smem, void *stream) {
    *grid = g_config.grid;
    *block = g_config.block;
    *smem = g_config.smem;
    *(cudaStream_t *)stream = g_config.stream;
    return cudaSuccess;
}
API cudaError_t cudaGetLastError() { return cudaSuccess; }
API const char *cudaGetErrorString(cudaError_t) { return "fake"; }
API cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t) { return cudaSuccess; }
API cudaError_t cudaMemcpyAsync(void *, const void *, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
API cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
API cudaError_t cudaGetSymbolAddress(void **p, const void *) {
    *p = g_area;
    return cudaSuccess;
}
API cudaError_t cudaGetDriverEntryPoint(const char *name, void **fn, unsigned long long,
                                        cudaDriverEntryPointQueryResult *q) {
    ++g_lookups;
    std::this_thread::sleep_for(std::chrono::milliseconds(200));  // long enough for another thread to arrive
    const bool known = !std::strcmp(name, "cuTensorMapEncodeTiled") && g_failing_lookups-- <= 0;
    *fn = known ? (void *)encode_tiled : nullptr;
    if (q) *q = known ? cudaDriverEntryPointSuccess : cudaDriverEntryPointSymbolNotFound;
    return cudaSuccess;
}

API void **__cudaRegisterFatBinary(void *) {
    static void *handle;
    return &handle;
}
API void __cudaRegisterFatBinaryEnd(void **) {}
API void __cudaUnregisterFatBinary(void **) {}
API void __cudaRegisterFunction(void **, const char *, char *, const char *, int, void *, void *, void *, void *,
                                int *) {}
API void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}
