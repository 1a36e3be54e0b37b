// rq_once.h -- launch attributes that are set once per device.
#pragma once

#include <atomic>
#include <cuda_runtime.h>

namespace rq {

// The function's dynamic shared memory, set once per device and function.
template <auto Kernel>
cudaError_t allow_smem(int bytes) {
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_relaxed);
    return e;
}

}  // namespace rq
