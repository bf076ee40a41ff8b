// Launch helpers: programmatic dependent launch, and the shared memory limit of a
// kernel raised once per device.
#pragma once

#include <atomic>

#include <cuda_runtime.h>
#include <stdint.h>

namespace nabla {

// Lets the dependent launch start once every CTA of this one has called it (or exited).
__device__ __forceinline__ void allow_dependents() {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
}
// Returns when the launches before have finished and their writes are visible.
__device__ __forceinline__ void wait_for_prerequisites() {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
}

}  // namespace nabla

// Host: a launch that may start while its predecessor in the stream still runs.
template <typename... P, typename... A>
inline cudaError_t nabla_launch_early(void (*kernel)(P...), unsigned grid, unsigned block, uint32_t smem,
                                      cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Host: dynamic shared memory of a kernel on the current device.  The attribute
// holds for the process; only the first call on a device sets it.  (Internal linkage:
// as an inline function its `set` would be one object for all copies of this library
// in a process, whose kernels each need the attribute.)
template <auto kKernel>
static cudaError_t nabla_allow_smem(uint32_t bytes) {
    static std::atomic<uint64_t> set{0};  // one bit a device
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if ((set.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
    err = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (err == cudaSuccess) set.fetch_or(bit, std::memory_order_release);
    return err;
}
