// Shared pieces of the row-norm kernels: a team of threads owns one row at a
// time.  Thread t of the team holds the 16-byte column vectors t, t + TPR,
// t + 2*TPR, ... of the row (VEC columns each), so consecutive lanes hold
// consecutive vectors: loads and stores are coalesced, and 128 neighbouring
// columns sit in 16 (16-bit storage) or 32 (fp32) neighbouring lanes.
//
// A team is 8 lanes, 16 (in the forward), a warp, or the whole CTA (TPR = 0).
//
// Rows that do not start on 16 bytes are held by the vectors of the aligned grid
// (SHIFT): vector v of a row has the columns v * VEC - shift .. + VEC - 1, where
// shift, the elements by which the row's start is past a 16-byte boundary, is
// the same in all tensors.  The vectors at a row's two ends also hold elements
// of its neighbours: they are read, not used and not written.  A team's rows are
// a multiple of VEC apart, so its shift, and with it the columns that a thread
// holds, stays the same over all of them.
//
// Tensors that are out of step with one another go by elements: thread t holds
// the columns t, t + TPR, t + 2*TPR, ..., so a warp's accesses are 64 or 128
// neighbouring bytes.
#pragma once

#include "dcn_common.cuh"
#include "dcn_tma.cuh"

namespace dcnb {

// NaN-propagating maximum (fmaxf drops NaN).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct SumOp {
    static __device__ __forceinline__ float apply(float a, float b) { return a + b; }
};
struct MaxOp {
    static __device__ __forceinline__ float apply(float a, float b) { return max_nan(a, b); }
};

template <typename OP, int W> __device__ __forceinline__ float lanes_reduce(float v) {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v = OP::apply(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Reduction over the team.  CTA teams go through `red` (two sets of 32 floats,
// used in turn, so one barrier per reduction is enough: a warp can be at most
// one reduction ahead of the slowest reader).
template <typename OP, int TPR> __device__ __forceinline__ float team_reduce(float v, float *red, int &turn) {
    if constexpr (TPR != 0) {
        return lanes_reduce<OP, TPR>(v);
    } else {
        v = lanes_reduce<OP, 32>(v);
        float *r = red + 32 * turn;
        turn ^= 1;
        const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) r[threadIdx.x >> 5] = v;
        __syncthreads();
        v = r[lane < nw ? lane : 0];
        if (lane >= nw) v = 0.0f;  // neutral: the sums and maxima here are of non-negative values or plain sums
        return lanes_reduce<OP, 32>(v);
    }
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t f2_bits(float2 a) { return *reinterpret_cast<uint64_t *>(&a); }
__device__ __forceinline__ float2 f2_fma(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
    return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float2 f2_mul(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(f2_bits(a)), "l"(f2_bits(b)));
    return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float2 f2_add(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(f2_bits(a)), "l"(f2_bits(b)));
    return *reinterpret_cast<float2 *>(&d);
}

// The VEC columns starting at column c of a row, as raw storage (zeros past the end).
template <typename T> __device__ __forceinline__ uint4 load_cols(const T *row, int c, int cols) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (c < cols) v = *reinterpret_cast<const uint4 *>(row + c);
    return v;
}

template <typename T> __device__ __forceinline__ void store_cols(T *row, int c, int cols, const uint4 &v) {
    if (c < cols) *reinterpret_cast<uint4 *>(row + c) = v;
}

// Elements by which the rows r0, r0 + a multiple of VEC, ... of a tensor start past a 16-byte boundary.
template <typename T> __device__ __forceinline__ int shift_of_rows(const void *base, long long r0, int cols) {
    constexpr int VEC = Storage<T>::kVec;
    return (int)(((reinterpret_cast<uintptr_t>(base) % 16) / sizeof(T) + (unsigned long long)r0 * cols) % VEC);
}

// The same for a vector of the aligned grid at columns c .. of the row at `off` in a tensor of `total` elements:
// whole, neighbours included, where it lies within the tensor.
template <typename T, bool SHIFT>
__device__ __forceinline__ uint4 load_vec(const T *base, long long off, int c, int cols, long long total) {
    constexpr int VEC = Storage<T>::kVec;
    if (!SHIFT) return load_cols<T>(base + off, c, cols);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (c >= cols) return v;
    if (off + c >= 0 && off + c + VEC <= total) return *reinterpret_cast<const uint4 *>(base + off + c);
    T e[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) e[j] = c + j >= 0 && c + j < cols ? base[off + c + j] : from_f32<T>(0.0f);
    memcpy(&v, e, 16);
    return v;
}

// A vector at any alignment, zeros outside the row.
template <typename T> __device__ __forceinline__ uint4 load_any(const T *row, int c, int cols) {
    constexpr int VEC = Storage<T>::kVec;
    T e[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) e[j] = c + j >= 0 && c + j < cols ? row[c + j] : from_f32<T>(0.0f);
    uint4 v;
    memcpy(&v, e, 16);
    return v;
}

// Bytes [b0, b1), all but not the whole, of a vector of 4 * W bytes whose elements have ES bytes, to the aligned `dst`:
// one store for each power of two that the part is made of, in which its two ends differ only by the places.
template <int W, int ES> __device__ __forceinline__ void store_part(void *dst, const uint32_t *w, int b0, int b1) {
    constexpr int S = 4 * W;
    unsigned char *p = static_cast<unsigned char *>(dst);
    auto word = [&](int at) {
        if constexpr (W == 1) return w[0];
        else if constexpr (W == 2) return at & 4 ? w[1] : w[0];
        else return at & 8 ? (at & 4 ? w[3] : w[2]) : (at & 4 ? w[1] : w[0]);
    };
    if (b0 > 0 && b1 < S) {
        // both ends in one vector: a row of fewer elements than it has
#pragma unroll
        for (int k = 0; k < S / ES; ++k) {
            if (k * ES < b0 || k * ES >= b1) continue;
            const uint32_t v = w[k * ES / 4] >> (8 * (k * ES % 4));
            if constexpr (ES == 4) *reinterpret_cast<uint32_t *>(p + k * ES) = v;
            else if constexpr (ES == 2) *reinterpret_cast<uint16_t *>(p + k * ES) = (uint16_t)v;
            else p[k] = (unsigned char)v;
        }
        return;
    }
    const bool head = b1 == S;  // a row's first vector: bytes from b0 on
    if constexpr (S > 8) {
        if (head ? b0 <= 8 : (b1 & 8) != 0) *reinterpret_cast<uint2 *>(p + (head ? 8 : 0)) = head ? make_uint2(w[2], w[3]) : make_uint2(w[0], w[1]);
    }
    if constexpr (S > 4) {
        const int at = head ? (b0 + 3) & ~3 : b1 & (S - 1) & ~7;
        if ((head ? at & 4 : b1 & 4) != 0) *reinterpret_cast<uint32_t *>(p + at) = word(at);
    }
    if constexpr (ES < 4) {
        const int at = head ? (b0 + 1) & ~1 : b1 & ~3;
        if ((head ? at & 2 : b1 & 2) != 0) *reinterpret_cast<uint16_t *>(p + at) = (uint16_t)(word(at) >> (8 * (at & 2)));
    }
    if constexpr (ES < 2) {
        const int at = head ? b0 : b1 & ~1;
        if ((head ? at & 1 : b1 & 1) != 0) p[at] = (unsigned char)(word(at) >> (8 * (at & 3)));
    }
}

// Only the row's own elements are written.
template <typename T, bool SHIFT> __device__ __forceinline__ void store_vec(T *row, int c, int cols, const uint4 &v) {
    constexpr int VEC = Storage<T>::kVec, ES = (int)sizeof(T);
    if (!SHIFT) {
        store_cols<T>(row, c, cols, v);
    } else if (c >= 0 && c + VEC <= cols) {
        *reinterpret_cast<uint4 *>(row + c) = v;
    } else if (c < cols) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        store_part<4, ES>(row + c, w, max(-c, 0) * ES, min(cols - c, VEC) * ES);
    }
}

// Ones over the elements of a vector that lie in the row.
template <typename T> __device__ __forceinline__ uint4 row_mask(int c, int cols) {
    constexpr int VEC = Storage<T>::kVec;
    uint32_t w[4] = {};
#pragma unroll
    for (int j = 0; j < VEC; ++j)
        if (c + j >= 0 && c + j < cols) w[j * 4 / VEC] |= VEC == 4 ? 0xffffffffu : 0xffffu << (16 * (j % 2));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 operator&(const uint4 &a, const uint4 &b) {
    return make_uint4(a.x & b.x, a.y & b.y, a.z & b.z, a.w & b.w);
}
// Zeros where a vector reaches out of its row.
template <typename T, bool SHIFT> __device__ __forceinline__ uint4 clear_outside(const uint4 &v, int c, int cols) {
    if (!SHIFT || (c >= 0 && c + Storage<T>::kVec <= cols)) return v;
    return v & row_mask<T>(c, cols);
}

// The staged vectors of a CTA team's rows.  Shifted, the first is vector 0 of thread 0 and the last, ragged one vector
// `last` of some thread.  KEEP: their masks are kept, all ones in the other threads, where there are registers for them;
// masks made row by row in the threads that need them hold the CTA up (fp16 5734 x 4383: backward 84 us against 73,
// forward 42.8 against 39.7; but to e4m3, which has no registers left, 49.8 against 52.5,
// before its codes were quotients).
template <typename T, bool SHIFT, bool KEEP> struct RowVecs {
    int cols;
    long long off;  // of the row in its tensor
    int shift = 0, nvec = 0, last = 0;
    bool ragged = false;  // a vector reaches out of the tensor, and was not staged
    long long total = 0;
    uint4 head, tail;
    __device__ __forceinline__ void init(int sh, int n, int t, int tpr) {
        if (!SHIFT) return;
        shift = sh;
        nvec = n;
        if (!KEEP) return;
        last = (n - 1) / tpr;
        head = row_mask<T>(t * Storage<T>::kVec - sh, cols);
        tail = row_mask<T>((t + last * tpr) * Storage<T>::kVec - sh, cols);
    }
    __device__ __forceinline__ void at(long long r, long long elems) {
        off = r * cols;
        if (!SHIFT) return;
        total = elems;
        ragged = off - shift < 0 || off - shift + (long long)nvec * Storage<T>::kVec > elems;
    }
    // vector i of the thread, at columns c ..
    __device__ __forceinline__ uint4 load(const unsigned char *row, const void *tensor, int i, int c) const {
        if (!SHIFT) return load_cols<T>(reinterpret_cast<const T *>(row), c, cols);
        if (ragged && c < cols && (off + c < 0 || off + c + Storage<T>::kVec > total))
            return load_any<T>(static_cast<const T *>(tensor) + off, c, cols);
        uint4 v = load_cols<T>(reinterpret_cast<const T *>(row) + shift, c, cols);
        if (!KEEP) return clear_outside<T, true>(v, c, cols);
        if (i == 0) v = v & head;
        if (i == last) v = v & tail;
        return v;
    }
};

// By elements: value k of a thread is column k * tpr + t.
template <typename T, int C> __device__ __forceinline__ void load_elems(const T *row, int t, int tpr, int cols, float *f) {
    T v[C];
#pragma unroll
    for (int k = 0; k < C; ++k) v[k] = k * tpr + t < cols ? row[k * tpr + t] : from_f32<T>(0.0f);
#pragma unroll
    for (int k = 0; k < C; ++k) f[k] = to_f32(v[k]);
}

// ---- rows staged in shared memory
//
// A team's rows are contiguous in memory, so one thread copies them by bulk
// asynchronous copies into a ring of slots, `slots` rows ahead; the team reads a
// slot once its barrier has counted the bytes and hands it back behind the
// barrier (or warp synchronisation) of the row's reduction.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

constexpr uint64_t kRowWaitNs = 1000000000ull;  // 1 s

// A wait for slot s ran out: reports it, and waits (again with a limit) for the other slots' copies in flight.
__device__ __forceinline__ void give_up(uint32_t bars, int s, uint32_t phase, int slots, unsigned int *err) {
    atomicOr(err, kDevErrTmaTimeout);
    for (int i = 1; i < slots; ++i) {
        const int k = s + i < slots ? s + i : s + i - slots;
        mbar_wait_bounded(bars + 8 * k, s + i < slots ? phase : phase ^ 1u, kRowWaitNs / 8);
    }
}

// Shared memory of the staged kernels: what a CTA may use when `ctas` of them share an SM (227 KB; the system takes
// 1 KB for each CTA, the kernels' barriers and sums another).
__host__ __device__ constexpr int staged_budget(int ctas) { return 227 * 1024 / ctas - 2048; }

}  // namespace dcnb
