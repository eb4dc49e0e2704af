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

// Least shared memory of a CTA that allocates `cols` columns of tensor memory, of `limit` bytes that a CTA may have.
// CTAs of a pair or a cluster wait for one another while they hold tensor memory.  Were a CTA that waits for its columns
// on an SM where others hold too many to get in the way of a cluster's last CTA there, two such clusters of calls on
// different streams could hold each other up for good.  So a CTA takes the same share of the shared memory as of the
// tensor memory: CTAs that fit an SM together find their columns there, and none waits.  All 512 columns leave 13 KB to
// CTAs without tensor memory: the smallest share of those with some is 14 KB.
// The fused core + projection keeps to half an SM's shared memory whatever its columns are (its gather lives on L1:
// 12800 pixels, 512 -> 512, 66.0 us so and 67.9 with its share), but waits for no other CTA.  It could only get in
// the way between two CTAs of clusters on its SM: a cluster's take a quarter at least, and two do not fit beside it.
inline size_t tensor_memory_share(size_t limit, int cols) {
    return cols >= 512 ? limit - 13 * 1024 : limit * cols / 512;
}

}  // namespace dcnb
