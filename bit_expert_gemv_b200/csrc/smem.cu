// Shared memory of the kernels that take more than 48 KB of it.
#include <cuda_runtime_api.h>

#include <mutex>

#include "gale.h"

namespace gale {

// Lets `kernel` be launched with up to `bytes` of dynamic shared memory on the
// current device.  Callers on several threads ask for sizes that differ from call
// to call: the limit is looked up, raised and recorded under one lock, and never
// lowered, so that a launch finds at least the limit that its caller asked for.
int ensure_smem(const void* kernel, int bytes) {
    constexpr int kMaxDev = 64, kMaxKernels = 64;      // (the library has fewer kernels)
    static const void* kernels[kMaxDev][kMaxKernels] = {};
    static int set_bytes[kMaxDev][kMaxKernels] = {};
    static std::mutex lock;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return GALE_ERR_CUDA;
    const std::lock_guard<std::mutex> held(lock);
    int slot = 0;
    while (slot < kMaxKernels && kernels[dev][slot] && kernels[dev][slot] != kernel) ++slot;
    if (slot == kMaxKernels) return GALE_ERR_CUDA;
    if (set_bytes[dev][slot] >= bytes) return GALE_OK;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return GALE_ERR_CUDA;
    kernels[dev][slot] = kernel;
    set_bytes[dev][slot] = bytes;
    return GALE_OK;
}

}  // namespace gale
