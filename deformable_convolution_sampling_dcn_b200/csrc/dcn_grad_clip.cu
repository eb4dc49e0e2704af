// Global gradient norm over many tensors, and clipping:
//   N = sqrt(sum g^2) or max |g| over all elements of all tensors
//   c = min(1, max_norm / (N + eps)),  out = rnd(g * c)
//
// The host hands the tensors over as a table in the kernel's parameters (no
// copy, no device allocation; a captured graph keeps it).  Tensors are cut
// into chunks of kChunk elements, aligned to 16 bytes of the gradient's own
// address, and the CTAs take chunks in turn.  The first kernel leaves one
// partial result per CTA, the second adds the partial results in a fixed
// order (no atomics: the norm is the same from run to run), derives c and
// rewrites the gradients.
//
// The squares of bf16 and fp32 gradients leave the range of fp32 (1e-23^2
// underflows, 1e20^2 overflows), so they are formed and summed in fp64; fp16
// squares and their per-thread sums fit fp32.
#include <math_constants.h>

#include "dcn_device.h"
#include "dcn_launch.h"
#include "dcn_norm.cuh"

namespace dcnb {
namespace {

constexpr int kChunk = 16384;      // elements
constexpr int kThreads = 256;
constexpr int kMaxCtas = 1184;     // 8 x 148

struct Entry {
    const void *g;
    void *out;
    int64_t n;           // elements
    uint32_t end_chunk;  // chunks of this and all earlier tensors of the table
    uint16_t gt, ot;     // DType of g and out
};

template <int CAP> struct Table {
    Entry e[CAP];
    int count;
};

constexpr int kSmallCap = 64, kLargeCap = 960;  // 2 KB and 30 KB of parameters (32764 bytes at most)

// Entry of chunk c.
template <int CAP> __device__ __forceinline__ int find_entry(const Table<CAP> &t, uint32_t c) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (t.e[mid].end_chunk <= c) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// Elements of storage type T that a chunk's grid is shifted by, so that its
// vectors sit on 16-byte boundaries of the gradient.
template <typename T> __host__ __device__ __forceinline__ int shift_of(const void *p) {
    return (int)((reinterpret_cast<uintptr_t>(p) % 16) / sizeof(T));
}

template <typename T> struct Acc {
    using type = double;
};
template <> struct Acc<__half> {
    using type = float;
};

// Partial result of elements [v0, v0 + kChunk) of the shifted grid.
template <typename T, bool INF> __device__ __forceinline__ double chunk_norm(const T *g, int64_t n, int64_t v0) {
    constexpr int VEC = Storage<T>::kVec;
    const int sh = shift_of<T>(g);
    const T *base = g - sh;  // 16-byte aligned; elements before g are never read
    typename Acc<T>::type s = 0;
    float m = 0.0f;
    const int64_t end = n + sh;
    for (int64_t v = v0 + threadIdx.x * VEC; v < v0 + kChunk && v < end; v += kThreads * VEC) {
        float f[VEC];
        if (v >= sh && v + VEC <= end) {
            unpack16<T>(*reinterpret_cast<const uint4 *>(base + v), f);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[j] = (v + j >= sh && v + j < end) ? to_f32(base[v + j]) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            if (INF) m = max_nan(m, fabsf(f[j]));
            else s += (typename Acc<T>::type)f[j] * (typename Acc<T>::type)f[j];
        }
    }
    return INF ? (double)m : (double)s;
}

__device__ __forceinline__ double combine(double a, double b, bool inf) {
    if (!inf) return a + b;
    return (a != a || b != b) ? CUDART_NAN : fmax(a, b);
}

__device__ __forceinline__ double cta_combine(double v, bool inf) {
    __shared__ double s[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = combine(v, __shfl_xor_sync(0xffffffffu, v, o), inf);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) v = combine(v, s[i], inf);
    return v;
}

template <int CAP, bool INF>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ Table<CAP> t, double *partial) {
    const uint32_t chunks = t.e[t.count - 1].end_chunk;
    double s = 0.0;
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int i = find_entry(t, c);
        const Entry &e = t.e[i];
        const int64_t v0 = (int64_t)(c - (i ? t.e[i - 1].end_chunk : 0)) * kChunk;
        double p;
        if (e.gt == (int)DType::F32) p = chunk_norm<float, INF>(static_cast<const float *>(e.g), e.n, v0);
        else if (e.gt == (int)DType::F16) p = chunk_norm<__half, INF>(static_cast<const __half *>(e.g), e.n, v0);
        else p = chunk_norm<__nv_bfloat16, INF>(static_cast<const __nv_bfloat16 *>(e.g), e.n, v0);
        s = combine(s, p, INF);
    }
    s = cta_combine(s, INF);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// The norm from the partial results, by every thread of a CTA.
__device__ __forceinline__ float total_norm(const double *partial, int n, bool inf) {
    double v = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) v = combine(v, partial[i], inf);
    v = cta_combine(v, inf);
    return (float)(inf ? v : sqrt(v));
}

__global__ void __launch_bounds__(kThreads) grad_norm_final_kernel(const double *partial, int n, int inf, float *norm) {
    const float v = total_norm(partial, n, inf != 0);
    if (threadIdx.x == 0) *norm = v;
}

template <typename T, typename O>
__device__ __forceinline__ void chunk_scale(const T *g, O *out, int64_t n, int64_t v0, float coef) {
    constexpr int VEC = Storage<T>::kVec, OV = Storage<O>::kVec;
    const int sh = shift_of<T>(g);
    const T *base = g - sh;
    O *obase = out - sh;
    const bool wide = reinterpret_cast<uintptr_t>(obase) % (VEC * sizeof(O) < 16 ? VEC * sizeof(O) : 16) == 0;
    const int64_t end = n + sh;
    for (int64_t v = v0 + threadIdx.x * VEC; v < v0 + kChunk && v < end; v += kThreads * VEC) {
        if (wide && v >= sh && v + VEC <= end) {
            float f[VEC];
            unpack16<T>(*reinterpret_cast<const uint4 *>(base + v), f);
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[j] *= coef;
            if constexpr (VEC >= OV) {
#pragma unroll
                for (int j = 0; j < VEC / OV; ++j)
                    reinterpret_cast<uint4 *>(obase + v)[j] = pack16<O>(f + j * OV);
            } else {  // fp32 gradients into 16-bit buffers: 8 bytes
                float h[OV] = {};
#pragma unroll
                for (int j = 0; j < VEC; ++j) h[j] = f[j];
                const uint4 p = pack16<O>(h);
                *reinterpret_cast<uint2 *>(obase + v) = make_uint2(p.x, p.y);
            }
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if (v + j >= sh && v + j < end) obase[v + j] = from_f32<O>(to_f32(base[v + j]) * coef);
        }
    }
}

template <typename T>
__device__ __forceinline__ void chunk_scale_to(const Entry &e, int64_t v0, float coef) {
    const T *g = static_cast<const T *>(e.g);
    if (e.ot == (int)DType::F32) chunk_scale<T, float>(g, static_cast<float *>(e.out), e.n, v0, coef);
    else if (e.ot == (int)DType::F16) chunk_scale<T, __half>(g, static_cast<__half *>(e.out), e.n, v0, coef);
    else chunk_scale<T, __nv_bfloat16>(g, static_cast<__nv_bfloat16 *>(e.out), e.n, v0, coef);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads)
    grad_scale_kernel(const __grid_constant__ Table<CAP> t, const double *partial, int n_partial, int inf,
                      float max_norm, float eps, float *norm, int write_norm) {
    const float total = total_norm(partial, n_partial, inf != 0);
    if (write_norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
    const float q = max_norm / (total + eps);
    const float coef = q > 1.0f ? 1.0f : q;  // a NaN norm gives NaN gradients
    const uint32_t chunks = t.e[t.count - 1].end_chunk;
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int i = find_entry(t, c);
        const Entry &e = t.e[i];
        // in place, a factor of one changes nothing
        if (coef == 1.0f && e.g == e.out && e.gt == e.ot) continue;
        const int64_t v0 = (int64_t)(c - (i ? t.e[i - 1].end_chunk : 0)) * kChunk;
        if (e.gt == (int)DType::F32) chunk_scale_to<float>(e, v0, coef);
        else if (e.gt == (int)DType::F16) chunk_scale_to<__half>(e, v0, coef);
        else chunk_scale_to<__nv_bfloat16>(e, v0, coef);
    }
}

size_t type_size(DType t) { return t == DType::F32 ? 4 : 2; }

uint32_t chunks_of(const ClipArgs &a, int i) {
    if (a.numel[i] == 0) return 0;
    const int64_t sh = (int64_t)((reinterpret_cast<uintptr_t>(a.grads[i]) % 16) / type_size((DType)a.dtypes[i]));
    return (uint32_t)((a.numel[i] + sh + kChunk - 1) / kChunk);
}

// Fills a table with the non-empty tensors from `first` on; returns the next tensor.
template <int CAP> int fill(const ClipArgs &a, int first, Table<CAP> &t) {
    t.count = 0;
    uint32_t end = 0;
    int i = first;
    for (; i < a.num_tensors && t.count < CAP; ++i) {
        const uint32_t c = chunks_of(a, i);
        if (!c) continue;
        Entry &e = t.e[t.count++];
        e.g = a.grads[i];
        e.out = a.outs ? a.outs[i] : const_cast<void *>(a.grads[i]);
        e.n = a.numel[i];
        end += c;
        e.end_chunk = end;
        e.gt = (uint16_t)a.dtypes[i];
        e.ot = (uint16_t)(a.outs ? a.out_dtypes[i] : a.dtypes[i]);
    }
    return i;
}

template <int CAP> int grid_of(const Table<CAP> &t) {
    const uint32_t c = t.e[t.count - 1].end_chunk;
    return (int)(c < (uint32_t)kMaxCtas ? c : (uint32_t)kMaxCtas);
}

template <int CAP> cudaError_t run(const ClipArgs &a, cudaStream_t stream) {
    static_assert(sizeof(Table<CAP>) + 64 <= 32764, "kernel parameters");
    Table<CAP> t;
    int n_partial = 0, tables = 0;
    for (int i = 0; i < a.num_tensors;) {
        i = fill(a, i, t);
        if (!t.count) break;
        const int grid = grid_of(t);
        if (a.inf) grad_norm_kernel<CAP, true><<<grid, kThreads, 0, stream>>>(t, a.partial + n_partial);
        else grad_norm_kernel<CAP, false><<<grid, kThreads, 0, stream>>>(t, a.partial + n_partial);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        n_partial += grid;
        ++tables;
    }
    if (!a.clip || !tables) {
        grad_norm_final_kernel<<<1, kThreads, 0, stream>>>(a.partial, n_partial, a.inf, a.norm);
        return cudaGetLastError();
    }
    int first = 1;
    for (int i = 0; i < a.num_tensors;) {
        if (tables > 1 || !first) i = fill(a, i, t);
        else i = a.num_tensors;  // the one table is still there
        if (!t.count) break;
        grad_scale_kernel<CAP><<<grid_of(t), kThreads, 0, stream>>>(t, a.partial, n_partial, a.inf, a.max_norm, a.eps,
                                                                  a.norm, first);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        first = 0;
    }
    return cudaSuccess;
}

}  // namespace

int64_t grad_clip_partials(int num_tensors) {
    const int64_t tables = ((int64_t)num_tensors + kLargeCap - 1) / kLargeCap;
    return (tables < 1 ? 1 : tables) * kMaxCtas;
}

cudaError_t launch_grad_clip(const ClipArgs &a, cudaStream_t stream) {
    int count = 0;
    for (int i = 0; i < a.num_tensors; ++i) count += a.numel[i] != 0;
    return count <= kSmallCap ? run<kSmallCap>(a, stream) : run<kLargeCap>(a, stream);
}

}  // namespace dcnb
