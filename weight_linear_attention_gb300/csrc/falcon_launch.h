// How the operators beside the scan are launched.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace falcon {

constexpr int kMaxDevices = 64;

// Launches kernel FN with programmatic stream serialisation: the launch overlaps the end of the kernel before it, so
// it waits (pdl_wait) before it reads or writes.
template <auto FN, typename... Args>
inline int launch_ahead(dim3 grid, int threads, int bytes, cudaStream_t s, Args... args) {
    if (bytes > 0) {
        static std::atomic<bool> ready[kMaxDevices];  // the kernel may have `bytes` of shared memory there
        int dev;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 4;
        if (!ready[dev].load(std::memory_order_acquire)) {
            if (cudaFuncSetAttribute(FN, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return 4;
            ready[dev].store(true, std::memory_order_release);
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, FN, args...) == cudaSuccess ? 0 : 4;
}

}  // namespace falcon
