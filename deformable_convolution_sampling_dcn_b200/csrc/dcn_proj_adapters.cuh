// Pieces shared by the kernels of the projection with low-rank adapters: the
// requests' row ranges and adapters, and the launch interface of the two
// routes (many rows: dcn_proj_adapters.cu, few rows: dcn_proj_adapters_rows.cu).
#pragma once

#include "dcn_common.cuh"
#include "dcn_host.h"
#include "dcn_launch.h"

namespace dcnb {

// Bit of the device error word: a request named an adapter outside [-1, num_adapters).
enum : unsigned { kDevErrBadAdapter = 2u };

constexpr int kMaxSmallRows = 256;  // columns of a tcgen05 product

// Adapter of request s: -1 for none.  An index out of range counts as none.
__device__ __forceinline__ int adapter_of(const int32_t *which, int s, int num_adapters) {
    const int a = which[s];
    return a >= 0 && a < num_adapters ? a : -1;
}

__device__ __forceinline__ void report_bad_adapter(int a, int num_adapters, unsigned int *err) {
    if (a < -1 || a >= num_adapters) atomicOr(err, kDevErrBadAdapter);
}

// First s of [0, n) for which pred(s) holds, which it then does up to n; n where there is none.  By a whole warp, 32
// places at a time: every step of a search in device memory is a round trip.
template <typename F> __device__ __forceinline__ int warp_first(int n, F pred) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;
    while (lo < hi) {
        const long long span = hi - lo;
        const unsigned hit = __ballot_sync(0xffffffffu, pred(lo + (int)(span * lane / 32)));
        const int i = hit ? __ffs((int)hit) - 1 : 32;  // the first of the places that holds: behind the one before it
        const int base = lo;
        if (i < 32) hi = base + (int)(span * i / 32);
        if (i > 0) lo = base + (int)(span * (i - 1) / 32) + 1;
    }
    return lo;
}

size_t adapters_small_workspace(const AdapterArgs &a);
size_t adapters_large_workspace(const AdapterArgs &a);
cudaError_t launch_adapters_small(const AdapterArgs &a, cudaStream_t stream);
cudaError_t launch_adapters_large(const AdapterArgs &a, cudaStream_t stream);

}  // namespace dcnb
