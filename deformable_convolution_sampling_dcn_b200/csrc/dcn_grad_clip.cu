// Global gradient norm over many tensors, and clipping:
//   N = sqrt(sum g^2) or max |g| over all elements of all tensors
//   c = min(1, max_norm / (N + eps)),  out = rnd(g * c)
//
// The host hands the tensors over as a table in the kernel's parameters (no
// copy, no device allocation; a captured graph keeps it).  Tensors are cut
// into chunks of 1024 16-byte vectors, four for each thread of a CTA, aligned
// to 16 bytes of the gradient's own address; every CTA takes a contiguous run
// of chunks, so it looks its first tensor up once and walks on from there.
// The first kernel leaves one partial result per CTA, the second adds the
// partial results in a fixed order (no atomics: the norm is the same from run
// to run), derives c and rewrites the gradients.
//
// Bound: device memory, the gradients being read twice.  The second pass walks
// the runs backwards and starts with what the first pass read last, of which L2
// still holds a part: of 194 MB of gradients 161 are read from device memory again.
// Measured (one B200): 301 bf16 tensors of 97 M elements into fp32
// 142 us, 34 us (5.7 TB/s) of it the norm; 13 fp32 tensors of 1.1 M elements 6.5
// us, two dependent launches.
//
// The squares of a vector (4 fp32, exact 8 of 16 bits) are added in fp32, the
// vectors in fp64.  Where that sum leaves [2^-90, 2^125) the squares are formed
// in fp64 instead: 1e-23^2 underflows fp32 and 1e20^2 overflows it.
#include <math_constants.h>

#include "dcn_device.h"
#include "dcn_launch.h"
#include "dcn_norm.cuh"

namespace dcnb {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;         // vectors of a thread in a chunk, all in flight at once
constexpr int kChunkVecs = kThreads * kUnroll;
// 6 CTAs on each of 148 SMs (the scaling's registers allow no more), in both passes: the second then starts where
// the first ended in every run.
constexpr int kMaxCtas = 888;

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

// The kUnroll vectors of this thread in the chunk that starts at vector q0 of the shifted grid.
template <typename T> __device__ __forceinline__ void load_chunk(const T *g, int64_t n, int64_t q0, uint4 *v) {
    constexpr int VEC = Storage<T>::kVec;
    const int sh = shift_of<T>(g);
    const T *base = g - sh;  // 16-byte aligned; elements before g and past its end are never read
    const int64_t end = n + sh;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const int64_t e = (q0 + i * kThreads + threadIdx.x) * VEC;
        v[i] = make_uint4(0, 0, 0, 0);
        if (e >= sh && e + VEC <= end) {
            v[i] = *reinterpret_cast<const uint4 *>(base + e);
        } else if (e < end) {
            T t[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) t[j] = e + j >= sh && e + j < end ? base[e + j] : from_f32<T>(0.0f);
            v[i] = *reinterpret_cast<uint4 *>(t);
        }
    }
}

// Partial result of a chunk.
template <typename T, bool INF> __device__ __forceinline__ double chunk_norm(const T *g, int64_t n, int64_t q0) {
    constexpr int VEC = Storage<T>::kVec;
    uint4 v[kUnroll];
    load_chunk<T>(g, n, q0, v);
    double s = 0.0;
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        float f[VEC];
        unpack16<T>(v[i], f);
        if (INF) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) m = max_nan(m, fabsf(f[j]));
        } else {
            float q = 0.0f;
#pragma unroll
            for (int j = 0; j < VEC; ++j) q = fmaf(f[j], f[j], q);
            if (q >= 0x1p-90f && q < 0x1p125f) {
                s += (double)q;
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) s += (double)f[j] * (double)f[j];
            }
        }
    }
    return INF ? (double)m : s;
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

// The chunks of CTA b of n: [chunks * b / n, chunks * (b + 1) / n).
__device__ __forceinline__ uint32_t run_begin(uint32_t chunks, uint32_t b, uint32_t n) {
    return (uint32_t)((uint64_t)chunks * b / n);
}

template <int CAP, bool INF>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ Table<CAP> t, double *partial) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t chunks = t.e[t.count - 1].end_chunk;
    const uint32_t c0 = run_begin(chunks, blockIdx.x, gridDim.x), c1 = run_begin(chunks, blockIdx.x + 1, gridDim.x);
    double s = 0.0;
    int i = find_entry(t, c0);
    for (uint32_t c = c0; c < c1; ++c) {
        while (t.e[i].end_chunk <= c) ++i;
        const Entry &e = t.e[i];
        const int64_t q0 = (int64_t)(c - (i ? t.e[i - 1].end_chunk : 0)) * kChunkVecs;
        double p;
        if (e.gt == (int)DType::F32) p = chunk_norm<float, INF>(static_cast<const float *>(e.g), e.n, q0);
        else if (e.gt == (int)DType::F16) p = chunk_norm<__half, INF>(static_cast<const __half *>(e.g), e.n, q0);
        else p = chunk_norm<__nv_bfloat16, INF>(static_cast<const __nv_bfloat16 *>(e.g), e.n, q0);
        s = combine(s, p, INF);
    }
    s = cta_combine(s, INF);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// The norm from the partial results, by every thread of a CTA.
__device__ __forceinline__ float total_norm(const double *partial, int n, bool inf) {
    double v = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) v = combine(v, __ldcg(partial + i), inf);
    v = cta_combine(v, inf);
    return (float)(inf ? v : sqrt(v));
}

__global__ void __launch_bounds__(kThreads) grad_norm_final_kernel(const double *partial, int n, int inf, float *norm) {
    const float v = total_norm(partial, n, inf != 0);
    if (threadIdx.x == 0) *norm = v;
}

// A vector's VEC products as storage type O: one store of 8, 16 or 32 bytes (whole sectors of L2 for a warp).
template <typename O, int VEC> __device__ __forceinline__ void store_vec(O *dst, const float *f) {
    constexpr int OV = Storage<O>::kVec;
    if constexpr (VEC == 2 * OV) {
        const uint4 lo = pack16<O>(f), hi = pack16<O>(f + OV);
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(lo.x), "r"(lo.y), "r"(lo.z),
                     "r"(lo.w), "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
                     : "memory");
    } else if constexpr (VEC == OV) {
        *reinterpret_cast<uint4 *>(dst) = pack16<O>(f);
    } else {
        float h[OV] = {};
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[j] = f[j];
        const uint4 p = pack16<O>(h);
        *reinterpret_cast<uint2 *>(dst) = make_uint2(p.x, p.y);
    }
}

template <typename T, typename O>
__device__ __forceinline__ void chunk_scale(const T *g, O *out, int64_t n, int64_t q0, float coef) {
    constexpr int VEC = Storage<T>::kVec, OB = VEC * (int)sizeof(O);  // bytes of a vector's store
    uint4 v[kUnroll];
    load_chunk<T>(g, n, q0, v);
    const int sh = shift_of<T>(g);
    const int64_t end = n + sh;
    const bool wide = (reinterpret_cast<uintptr_t>(out) - sh * sizeof(O)) % OB == 0;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const int64_t e = (q0 + i * kThreads + threadIdx.x) * VEC;
        if (e >= end) break;
        float f[VEC];
        unpack16<T>(v[i], f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] *= coef;
        O *dst = out + (e - sh);
        if (wide && e >= sh && e + VEC <= end) {
            store_vec<O, VEC>(dst, f);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if (e + j >= sh && e + j < end) dst[j] = from_f32<O>(f[j]);
        }
    }
}

template <typename T> __device__ __forceinline__ void chunk_scale_to(const Entry &e, int64_t q0, float coef) {
    const T *g = static_cast<const T *>(e.g);
    if (e.ot == (int)DType::F32) chunk_scale<T, float>(g, static_cast<float *>(e.out), e.n, q0, coef);
    else if (e.ot == (int)DType::F16) chunk_scale<T, __half>(g, static_cast<__half *>(e.out), e.n, q0, coef);
    else chunk_scale<T, __nv_bfloat16>(g, static_cast<__nv_bfloat16 *>(e.out), e.n, q0, coef);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, 6)
    grad_scale_kernel(const __grid_constant__ Table<CAP> t, const double *partial, int n_partial, int inf,
                      float max_norm, float eps, float *norm, int write_norm) {
    const uint32_t chunks = t.e[t.count - 1].end_chunk;
    const uint32_t c0 = run_begin(chunks, blockIdx.x, gridDim.x), c1 = run_begin(chunks, blockIdx.x + 1, gridDim.x);
    int i = find_entry(t, c1 - 1);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial results
    const float total = total_norm(partial, n_partial, inf != 0);
    if (write_norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
    const float q = max_norm / (total + eps);
    const float coef = q > 1.0f ? 1.0f : q;  // a NaN norm gives NaN gradients
    for (uint32_t c = c1; c-- > c0;) {
        while (i && t.e[i - 1].end_chunk > c) --i;
        const Entry &e = t.e[i];
        // in place, a factor of one changes nothing
        if (coef == 1.0f && e.g == e.out && e.gt == e.ot) continue;
        const int64_t q0 = (int64_t)(c - (i ? t.e[i - 1].end_chunk : 0)) * kChunkVecs;
        if (e.gt == (int)DType::F32) chunk_scale_to<float>(e, q0, coef);
        else if (e.gt == (int)DType::F16) chunk_scale_to<__half>(e, q0, coef);
        else chunk_scale_to<__nv_bfloat16>(e, q0, coef);
    }
}

size_t type_size(DType t) { return t == DType::F32 ? 4 : 2; }

uint32_t chunks_of(const ClipArgs &a, int i) {
    if (a.numel[i] == 0) return 0;
    const int64_t es = (int64_t)type_size((DType)a.dtypes[i]);
    const int64_t bytes = a.numel[i] * es + (int64_t)(reinterpret_cast<uintptr_t>(a.grads[i]) % 16);
    return (uint32_t)((bytes + kChunkVecs * 16 - 1) / (kChunkVecs * 16));
}

// Fills a table with the non-empty tensors from `first` on; returns the next non-empty tensor (a table is empty only
// where there is none at all), num_tensors behind the last.
template <int CAP> int fill(const ClipArgs &a, int first, Table<CAP> &t) {
    t.count = 0;
    uint32_t end = 0;
    int i = first;
    for (; i < a.num_tensors; ++i) {
        const uint32_t c = chunks_of(a, i);
        if (!c) continue;
        if (t.count == CAP) break;
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
        // a programmatic dependent: it reads nothing that the norm kernel writes before its wait, and writes
        // nothing before it either
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)grid_of(t));
        cfg.blockDim = dim3(kThreads);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, grad_scale_kernel<CAP>, t, (const double *)a.partial, n_partial,
                                                 (int)a.inf, a.max_norm, a.eps, a.norm, first);
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
