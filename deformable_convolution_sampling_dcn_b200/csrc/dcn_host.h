// Host-side helpers of the launchers.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace dcnb {

// Lets `kern` use `bytes` of shared memory, once per device; `done` is the kernel's own array of flags.
constexpr int kMaxDev = 64;
template <typename K> cudaError_t allow_smem(K kern, int bytes, std::atomic<bool> (&done)[kMaxDev]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDev && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev >= 0 && dev < kMaxDev) done[dev].store(true, std::memory_order_release);
    return e;
}

}  // namespace dcnb
