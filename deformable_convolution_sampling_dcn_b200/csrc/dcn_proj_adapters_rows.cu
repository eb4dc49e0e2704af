// Projection with low-rank adapters, few rows (at most 64): single tokens of
// many requests.
//   t[m, :] = scale[a] * A[a] x[m]             a = adapter of row m's request
//   y[m, n] = bias[n] + sum_k W[n, k] x[m, k] + sum_j B[a][n, j] t[m, j]
//
// Bound: the weight, which is read once whatever the rows are.
//
// The first kernel forms t (fp32, never rounded) with one warp per (row, rank)
// and leaves it, with each row's adapter, in the workspace.  The second starts
// at the same time (programmatic dependent launch) and needs t only in its
// epilogue.  A cluster of CTAs owns 128 output channels and splits the
// contraction; each warp takes 16 channels and multiplies its slice of the
// weight, straight from device memory, with all rows by mma.sync (the rows are
// the narrow dimension: a 128-row tcgen05 tile would be mostly padding, and
// the kernel waits for memory, not for the products).  The order of the
// contraction is free, so lane (g, q) loads 8 neighbouring channels of weight
// row g and of x row g with one 16-byte load each and uses them as the
// fragments of two products.  The cluster's CTAs leave their fp32 partial sums
// in shared memory, and each adds up its share of the rows through distributed
// shared memory.
#include <cooperative_groups.h>

#include "dcn_device.h"
#include "dcn_proj_adapters.cuh"

namespace dcnb {
namespace {

namespace cg = cooperative_groups;

constexpr int kRowThreads = 256;
constexpr int kRowN = 128;  // output channels of a cluster: 8 warps x 16

struct SmallParams {
    AdapterArgs a;
    float *t;             // [rows, rank]
    int32_t *row_adapter; // [rows]: adapter, -1 none, -2 the row belongs to no request
    unsigned int *err;
    int k_slice;          // channels of a CTA's part of the contraction, a multiple of 32
};

template <typename T>
__global__ void __launch_bounds__(kRowThreads) adapters_rows_shrink(const SmallParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const AdapterArgs &a = p.a;
    const int m = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // requests that end at or before row m, and whether the first one starts after it
    int before = 0;
    for (int s = threadIdx.x; s < a.requests; s += kRowThreads) before += a.start[s + 1] <= m;
    before = __reduce_add_sync(0xffffffffu, before);
    __shared__ int sums[kRowThreads / 32];
    if (lane == 0) sums[warp] = before;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int i = 0; i < kRowThreads / 32; ++i) s += sums[i];
    const bool covered = s < a.requests && a.start[s < a.requests ? s : 0] <= m;
    const int ad = covered ? adapter_of(a.which, s, a.adapters) : -1;
    if (blockIdx.y == 0 && threadIdx.x == 0) {
        p.row_adapter[m] = covered ? ad : -2;
        if (covered) report_bad_adapter(a.which[s], a.adapters, p.err);
    }
    const int r = blockIdx.y * (kRowThreads / 32) + warp;
    if (ad < 0 || r >= a.rank) return;
    const T *x = static_cast<const T *>(a.x) + (long long)m * a.cin;
    const T *w = static_cast<const T *>(a.a) + ((long long)ad * a.rank + r) * a.cin;
    float acc = 0.0f;
#pragma unroll 4
    for (int k = lane * 8; k < a.cin; k += 256) {
        float f[8], g[8];
        unpack16<T>(ld_nc16(x + k), f);
        unpack16<T>(ld_nc16(w + k), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc = fmaf(f[j], g[j], acc);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) p.t[(long long)m * a.rank + r] = acc * (a.scale ? a.scale[ad] : 1.0f);
}

template <typename T>
__device__ __forceinline__ void mma_16816(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1);
template <>
__device__ __forceinline__ void mma_16816<__half>(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                  uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma_16816<__nv_bfloat16>(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes of row `row` (of `rows`) from column k, zeros outside.
template <typename T>
__device__ __forceinline__ uint4 load_frag(const T *base, int row, int rows, int k, int k_end, long long ld) {
    if (row >= rows || k >= k_end) return make_uint4(0, 0, 0, 0);
    return ld_nc16(base + (long long)row * ld + k);
}

// MT tiles of 8 rows; the cluster's CTAs (blockIdx.x) split the contraction.
template <typename T, int MT>
__global__ void __launch_bounds__(kRowThreads) adapters_rows_project(const SmallParams p) {
    extern __shared__ float part[];  // [MT * 8][kRowN]
    cg::cluster_group cluster = cg::this_cluster();
    const AdapterArgs &a = p.a;
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int n0 = blockIdx.y * kRowN, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, q = lane & 3;
    const T *x = static_cast<const T *>(a.x), *w = static_cast<const T *>(a.weight);
    const int rows = (int)a.rows;
    const int k0 = rank * p.k_slice, k1 = min(a.cin, k0 + p.k_slice);
    const int n = n0 + warp * 16 + g;

    float acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
#pragma unroll 4
    for (int k = k0 + q * 8; k < k1 + q * 8; k += 32) {
        const uint4 w0 = load_frag(w, n, a.cout, k, k1, a.cin), w1 = load_frag(w, n + 8, a.cout, k, k1, a.cin);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const uint4 xv = load_frag(x, i * 8 + g, rows, k, k1, a.cin);
            mma_16816<T>(acc[i], w0.x, w1.x, w0.y, w1.y, xv.x, xv.y);
            mma_16816<T>(acc[i], w0.z, w1.z, w0.w, w1.w, xv.z, xv.w);
        }
    }
    // accumulator element (channel g or g + 8, rows 2q and 2q + 1 of the tile)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            part[(i * 8 + 2 * q + (j & 1)) * kRowN + warp * 16 + g + (j >= 2 ? 8 : 0)] = acc[i][j];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // t and row_adapter of the first kernel
    cluster.sync();

    const int c = threadIdx.x % kRowN, o = n0 + c;
    const T *bias = static_cast<const T *>(a.bias);
    T *out = static_cast<T *>(a.out);
    const float b0 = bias && o < a.cout ? to_f32(bias[o]) : 0.0f;
    for (int m = rank + ranks * (threadIdx.x / kRowN); m < rows; m += ranks * (kRowThreads / kRowN)) {
        float v = 0.0f;
        for (int s = 0; s < ranks; ++s) v += cluster.map_shared_rank(part, s)[m * kRowN + c];
        const int ad = __ldcg(p.row_adapter + m);
        if (ad >= 0 && o < a.cout) {
            const T *b = static_cast<const T *>(a.b) + ((long long)ad * a.cout + o) * a.rank;
            const float *t = p.t + (long long)m * a.rank;
            float u = 0.0f;
            for (int j = 0; j < a.rank; j += 8) {
                float f[8];
                unpack16<T>(ld_nc16(b + j), f);
                const float4 t0 = __ldcg(reinterpret_cast<const float4 *>(t + j));
                const float4 t1 = __ldcg(reinterpret_cast<const float4 *>(t + j + 4));
                u = fmaf(f[0], t0.x, u); u = fmaf(f[1], t0.y, u); u = fmaf(f[2], t0.z, u); u = fmaf(f[3], t0.w, u);
                u = fmaf(f[4], t1.x, u); u = fmaf(f[5], t1.y, u); u = fmaf(f[6], t1.z, u); u = fmaf(f[7], t1.w, u);
            }
            v += u;
        }
        if (ad != -2 && o < a.cout) out[(long long)m * a.cout + o] = from_f32<T>(v + b0);
    }
    cluster.sync();  // the other CTAs may still read this one's partial sums
}

template <typename T, int MT> cudaError_t launch_mt(const SmallParams &p, int ranks, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ranks, (unsigned)((p.a.cout + kRowN - 1) / kRowN));
    cfg.blockDim = dim3(kRowThreads);
    cfg.dynamicSmemBytes = (size_t)MT * 8 * kRowN * sizeof(float);  // at most 32 KB
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, adapters_rows_project<T, MT>, p);
}

template <typename T> cudaError_t launch_t(const AdapterArgs &a, cudaStream_t stream) {
    const DeviceInfo *dev = device_info();
    if (!dev) return cudaErrorNotSupported;
    SmallParams p;
    p.a = a;
    p.t = static_cast<float *>(a.workspace);
    p.row_adapter = reinterpret_cast<int32_t *>(p.t + a.rows * a.rank);
    p.err = dev->err;
    const int nt = (a.cout + kRowN - 1) / kRowN;
    // split the contraction until there are two CTAs for every SM, down to 64 channels a CTA
    int ranks = 1;
    while (ranks < 8 && nt * ranks < 2 * dev->sms && a.cin / (2 * ranks) >= 64) ranks *= 2;
    p.k_slice = ((a.cin + ranks - 1) / ranks + 31) / 32 * 32;
    adapters_rows_shrink<T><<<dim3((unsigned)a.rows, (unsigned)((a.rank + 7) / 8)), kRowThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (a.rows <= 8) return launch_mt<T, 1>(p, ranks, stream);
    if (a.rows <= 16) return launch_mt<T, 2>(p, ranks, stream);
    if (a.rows <= 32) return launch_mt<T, 4>(p, ranks, stream);
    return launch_mt<T, 8>(p, ranks, stream);
}

}  // namespace

size_t adapters_small_workspace(const AdapterArgs &a) { return (size_t)a.rows * a.rank * 4 + (size_t)a.rows * 4; }

cudaError_t launch_adapters_small(const AdapterArgs &a, cudaStream_t stream) {
    switch (a.dtype) {
        case DType::F16: return launch_t<__half>(a, stream);
        case DType::BF16: return launch_t<__nv_bfloat16>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace dcnb
