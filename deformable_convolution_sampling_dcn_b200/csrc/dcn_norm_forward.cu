// Residual addition and root-mean-square norm, with the output in the storage
// type, in 8 bits with scales, or both:
//   h    = rnd(x + residual)             (h = x without a residual)
//   rstd = 1 / sqrt(mean_c(h^2) + eps)
//   y    = h * rstd * weight
//   8 bit: s = max(max|y| / top, 2^-126) over the row or over 128 columns,
//          q = rnd(y / s), top = 448 (e4m3) or 127 (int8)
// h is rounded to the storage type first because that is the value the next
// block's residual and the backward pass read; everything after it is fp32 and
// rounded once.
//
// Bound: device memory.  One pass: a row stays in the registers of its team
// between the statistics and the output, so each byte moves once.  Measured (one
// B200): bf16 102400 x 256 with a residual 34.4 us (210 MB: 6.1 TB/s of 6.56),
// fp16 12800 x 512 to e4m3 9.8 us (46 MB: 4.7 TB/s), bf16 2047 x 4096 to int8 in
// groups 14.9 us (59 MB: 4.0 TB/s); off 16-byte boundaries fp16 5734 x 4383 with a
// residual 39.7 us (201 MB: 5.1 TB/s), to int8 in groups 64 us, where the
// instructions bound it.
#include <cuda_fp8.h>

#include "dcn_device.h"
#include "dcn_host.h"
#include "dcn_launch.h"
#include "dcn_norm.cuh"

namespace dcnb {
namespace {

constexpr float kScaleMin = 1.17549435e-38f;  // 2^-126: a normal number, an all-zero row gives q = 0

// Four values times `f` to four 8-bit codes, in memory order.  int8 rounds by
// adding 1.5 * 2^23 in the fused product: the low byte of the sum is the rounded
// value (|v * f| <= 127 * (1 + 2^-20)).
__device__ __forceinline__ uint32_t pack8(float2 v0, float2 v1, float f, int quant) {
    const float2 ff = make_float2(f, f);
    if (quant == kQuantE4M3) {
        const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(f2_mul(v0, ff), __NV_SATFINITE, __NV_E4M3);
        const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(f2_mul(v1, ff), __NV_SATFINITE, __NV_E4M3);
        return (uint32_t)lo | ((uint32_t)hi << 16);
    }
    const float2 round = make_float2(12582912.0f, 12582912.0f);
    const float2 q0 = f2_fma(v0, ff, round), q1 = f2_fma(v1, ff, round);
    return __byte_perm(__byte_perm(__float_as_uint(q0.x), __float_as_uint(q0.y), 0x0040),
                       __byte_perm(__float_as_uint(q1.x), __float_as_uint(q1.y), 0x0040), 0x5410);
}

// A code is the quotient y / s, divided in fp32 and rounded once more.  A product
// with 1 / s is off by up to 1.5 steps of fp32, which puts some values on the other
// side of a border between two codes; but a product 2^-21 below it and one as far
// above have the quotient between them, so where both give the same code it is the
// quotient's (rounding is monotonic), and only the others, a vector in some ten
// thousand, divide.  (bf16 2047 x 4096 to int8: 14.8 us, 13.7 with the products alone,
// 16.4 with divisions alone.)
constexpr float kBelow = 1.0f - 0x1p-21f, kAbove = 1.0f + 0x1p-21f;

// A scale and its inverse.
struct Scale {
    float s, inv;
};
__device__ __forceinline__ Scale with_inverse(float s) { return {s, 1.0f / s}; }

// The codes of N values (a multiple of 4), the first `lo` (SHIFT) with the scale `before`, the others with `s`.
template <int N, bool SHIFT>
__device__ __forceinline__ void codes_of(const float *y, Scale s, Scale before, int lo, int quant, uint32_t *q) {
    const float below = SHIFT ? kBelow : s.inv * kBelow, above = SHIFT ? kAbove : s.inv * kAbove;
    uint32_t differ = 0;
    if constexpr (SHIFT) {
#pragma unroll
        for (int k = 0; k < N / 4; ++k) {
            float2 v[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = 4 * k + 2 * i;
                v[i] = f2_mul(make_float2(y[j], y[j + 1]), make_float2(j < lo ? before.inv : s.inv, j + 1 < lo ? before.inv : s.inv));
            }
            q[k] = pack8(v[0], v[1], below, quant);
            differ |= q[k] ^ pack8(v[0], v[1], above, quant);
        }
    } else {
#pragma unroll
        for (int k = 0; k < N / 4; ++k) {
            const float2 v0 = make_float2(y[4 * k], y[4 * k + 1]), v1 = make_float2(y[4 * k + 2], y[4 * k + 3]);
            q[k] = pack8(v0, v1, below, quant);
            differ |= q[k] ^ pack8(v0, v1, above, quant);
        }
    }
    if (differ) {
#pragma unroll
        for (int k = 0; k < N / 4; ++k) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = y[4 * k + i] / (SHIFT && 4 * k + i < lo ? before.s : s.s);
            q[k] = pack8(make_float2(v[0], v[1]), make_float2(v[2], v[3]), 1.0f, quant);
        }
    }
}

// The same for one value.
__device__ __forceinline__ unsigned char code1(float v, float f, int quant) {
    if (quant == kQuantE4M3) return __nv_cvt_float_to_fp8(v * f, __NV_SATFINITE, __NV_E4M3);
    return (unsigned char)__float_as_uint(fmaf(v, f, 12582912.0f));
}
__device__ __forceinline__ unsigned char code_of(float y, Scale s, int quant) {
    const unsigned char q = code1(y, s.inv * kBelow, quant);
    return q == code1(y, s.inv * kAbove, quant) ? q : code1(y / s.s, 1.0f, quant);
}

// The codes of a thread's vector at columns c ..; row + c is a multiple of VEC.  The first `lo` elements have the
// scale `before`, the others `s`.
template <int VEC, bool SHIFT>
__device__ __forceinline__ void store_codes(unsigned char *row, int c, int cols, const float *y, Scale s, Scale before,
                                            int lo, int quant) {
    if (c >= cols) return;
    uint32_t q[VEC / 4];
    codes_of<VEC, SHIFT>(y, s, before, lo, quant, q);
    if (!SHIFT || (c >= 0 && c + VEC <= cols)) {
        if constexpr (VEC == 8) *reinterpret_cast<uint2 *>(row + c) = make_uint2(q[0], q[1]);
        else *reinterpret_cast<uint32_t *>(row + c) = q[0];
    } else {
        store_part<VEC / 4, 1>(row + c, q, max(-c, 0), min(cols - c, VEC));
    }
}

// Largest magnitude of a vector's elements from `lo` on, and into `before` of those ahead.  Elements outside the row
// hold 0 * rstd * 0: zero, or NaN where every element of the row is.
template <int VEC, bool SHIFT> __device__ __forceinline__ float vec_max(const float *y, int lo, float &before) {
    float m = 0.0f;
    before = 0.0f;
    if (SHIFT && lo) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            before = max_nan(before, j < lo ? fabsf(y[j]) : 0.0f);
            m = max_nan(m, j < lo ? 0.0f : fabsf(y[j]));
        }
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) m = max_nan(m, fabsf(y[j]));
    }
    return m;
}

__device__ __forceinline__ float scale_of(float amax, int quant) {
    return max_nan(amax / (quant == kQuantE4M3 ? 448.0f : 127.0f), kScaleMin);
}

constexpr int kMaxSlots = 8;

// Teams of 8, 16 and 32 lanes in CTAs of 256 threads.  A thread holds C = NV * VEC
// columns of a row: up to two vectors with the loads of its team's next row in
// flight meanwhile, or four without (which fp32 has the registers for, but only
// with spills: 40000 x 304 to e4m3 58 us against 31); CTAs on an SM follow from
// the registers that leaves (64, 80 or 128).
constexpr int kTeamThreads = 256;
constexpr int ctas_per_sm(int c) { return c <= 8 ? 4 : c <= 16 ? 3 : 2; }

template <typename T, int TPR, int NV, bool QUANT, bool SHIFT>
__global__ void __launch_bounds__(kTeamThreads, ctas_per_sm(NV * Storage<T>::kVec))
    norm_forward_kernel(const NormArgs a) {
    constexpr int VEC = Storage<T>::kVec;
    constexpr bool AHEAD = NV <= 2;
    constexpr int tpr = TPR, teams = kTeamThreads / TPR;  // teams: a multiple of VEC
    const int t = (int)threadIdx.x % TPR, team = (int)threadIdx.x / TPR;
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    const T *weight = static_cast<const T *>(a.weight);
    const long long total = a.rows * a.cols;
    const int sh = SHIFT ? shift_of_rows<T>(a.x, (long long)blockIdx.x * teams + team, a.cols) : 0;
    auto column = [&](int i) { return (t + i * tpr) * VEC - sh; };
    uint4 w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (weight) w[i] = SHIFT ? load_any<T>(weight, column(i), a.cols) : load_cols<T>(weight, column(i), a.cols);
    uint4 keep[NV];
    constexpr bool KEEP = SHIFT && NV <= 2;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (KEEP) keep[i] = row_mask<T>(column(i), a.cols);
    auto own = [&](const uint4 &v, int i) {
        return !SHIFT ? v : KEEP ? v & keep[i] : clear_outside<T, SHIFT>(v, column(i), a.cols);
    };

    uint4 xn[NV], rn[NV];
    auto fetch = [&](long long r) {
        const long long off = r < a.rows ? r * a.cols : 0;
        const int cols = r < a.rows ? a.cols : 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            xn[i] = load_vec<T, SHIFT>(x, off, column(i), cols, total);
            if (res) rn[i] = load_vec<T, SHIFT>(res, off, column(i), cols, total);
        }
    };
    const long long step = (long long)gridDim.x * teams;
    if (AHEAD) fetch((long long)blockIdx.x * teams + team);
    // every lane of a warp runs the same number of rounds: the shuffles need them all
    for (long long base = (long long)blockIdx.x * teams; base < a.rows; base += step) {
        const long long r = base + team;
        const bool live = r < a.rows;
        const long long off = live ? r * a.cols : 0;
        const int cols = live ? a.cols : 0;
        if (!AHEAD) fetch(r);
        float y[NV][VEC];
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack16<T>(own(xn[i], i), y[i]);
            if (res) {
                float g[VEC];
                unpack16<T>(own(rn[i], i), g);
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[i][j] += g[j];
                const uint4 h = pack16<T>(y[i]);
                store_vec<T, SHIFT>(static_cast<T *>(a.residual_out) + off, column(i), cols, h);
                unpack16<T>(h, y[i]);
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) ss = fmaf(y[i][j], y[i][j], ss);
        }
        if (AHEAD) fetch(r + step);
        ss = lanes_reduce<SumOp, TPR>(ss);
        const float rstd = 1.0f / sqrtf(ss / (float)a.cols + a.eps);
        if (a.rstd && t == 0 && live) a.rstd[r] = rstd;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (weight) {
                float g[VEC];
                unpack16<T>(w[i], g);
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[i][j] = y[i][j] * rstd * g[j];
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[i][j] *= rstd;
            }
            if (!QUANT || a.out)
                store_vec<T, SHIFT>(static_cast<T *>(a.out) + off, column(i), cols, pack16<T>(y[i]));
        }
        if constexpr (QUANT) {
            // lanes that share 128 columns; teams narrower than a warp hold rows of at most 128 columns
            constexpr int GL = 128 / VEC;
            const bool grouped = a.group != 0 && TPR == 32;
            // of shifted vectors the first of a group also holds the end of the group before
            float gmax[NV], before[NV], amax = 0.0f, s[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                gmax[i] = vec_max<VEC, SHIFT>(y[i], grouped && t % GL == 0 ? sh : 0, before[i]);
                amax = max_nan(amax, gmax[i]);
            }
            if (!grouped) {
                s[0] = scale_of(lanes_reduce<MaxOp, TPR>(amax), a.quant);
                if (t == 0 && live) a.scale[r] = s[0];
#pragma unroll
                for (int i = 1; i < NV; ++i) s[i] = s[0];
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float m = lanes_reduce<MaxOp, (GL < 32 ? GL : 32)>(gmax[i]);
                    if (SHIFT) {
                        const float here = __shfl_sync(0xffffffffu, before[i], 16);
                        const float next = i + 1 < NV ? __shfl_sync(0xffffffffu, before[i + 1 < NV ? i + 1 : i], 0) : 0.0f;
                        m = max_nan(m, GL == 16 && t < 16 ? here : next);
                    }
                    s[i] = scale_of(m, a.quant);
                    const int v = t + i * tpr;
                    if (v % GL == 0 && v * VEC < cols) a.scale[r * a.groups + v / GL] = s[i];
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                Scale s0 = {};
                if (SHIFT && grouped) {
                    const float here = __shfl_sync(0xffffffffu, s[i], 15);
                    const float last = __shfl_sync(0xffffffffu, s[i ? i - 1 : 0], 31);
                    if (t % GL == 0) s0 = with_inverse(GL == 16 && t == 16 ? here : last);
                }
                store_codes<VEC, SHIFT>(static_cast<unsigned char *>(a.out8) + off, column(i), cols, y[i], with_inverse(s[i]), s0,
                                        grouped && t % GL == 0 ? sh : 0, a.quant);
            }
        }
    }
}

// Rows wider than a warp team holds: a CTA of 16 columns a thread per row, the
// rows staged by bulk copies (bf16 2047 x 4096 to int8: 16.8 us with the next
// row's loads in registers, 14.0 us staged, before the codes were quotients).  A shifted row's groups of 128
// columns begin inside vectors, so their maxima meet in shared memory.
template <typename T, bool QUANT, bool SHIFT>
__global__ void __launch_bounds__(1024, 1) norm_forward_wide_kernel(const NormArgs a, int slots, unsigned int *err) {
    constexpr int VEC = Storage<T>::kVec, NV = 16 / VEC, GL = 128 / VEC;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ float red[64];
    __shared__ __align__(8) uint64_t bars[kMaxSlots];
    // shifted rows: maxima of the groups (bits of values >= 0) and the scales that follow from them, with their inverses
    __shared__ int gmax_s[QUANT && SHIFT ? 128 : 1];
    __shared__ Scale scale_s[QUANT && SHIFT ? 128 : 1];
    const int t = threadIdx.x, tpr = blockDim.x;
    const T *weight = static_cast<const T *>(a.weight);
    const long long step = gridDim.x, total = a.rows * a.cols;  // SHIFT: step is a multiple of VEC, or no CTA has two rows
    const int sh = SHIFT ? shift_of_rows<T>(a.x, blockIdx.x, a.cols) : 0, nvec = (a.cols + sh + VEC - 1) / VEC;
    // a row in the ring: its vectors of the aligned grid, without one that reaches out of the tensor at either end
    const uint32_t row_bytes = (uint32_t)nvec * 16, slot_bytes = a.residual ? 2 * row_bytes : row_bytes;
    int turn = 0;
    if (t == 0) {
        for (int i = 0; i < slots; ++i) mbar_init(smem_u32(bars + i), 1);
        fence_mbar_init();
    }
    if (QUANT && SHIFT)
        for (int i = t; i < 128; i += tpr) gmax_s[i] = 0;
    __syncthreads();
    auto stage = [&](long long r, int s) {  // by thread 0
        if (r >= a.rows) return;
        const long long e = r * a.cols - sh;
        const int skip = SHIFT && e < 0, n = nvec - skip - (SHIFT && e + (long long)nvec * VEC > total);
        const uint32_t bar = smem_u32(bars + s), dst = smem_u32(ring) + s * slot_bytes + 16 * skip;
        mbar_arrive_expect_tx(bar, (a.residual ? 32u : 16u) * n);
        bulk_load(dst, static_cast<const T *>(a.x) + e + skip * VEC, 16u * n, bar);
        if (a.residual) bulk_load(dst + row_bytes, static_cast<const T *>(a.residual) + e + skip * VEC, 16u * n, bar);
    };
    if (t == 0)
        for (int i = 0; i < slots; ++i) stage(blockIdx.x + i * step, i);
    auto column = [&](int i) { return (t + i * tpr) * VEC - sh; };
    uint4 w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (weight) w[i] = SHIFT ? load_any<T>(weight, column(i), a.cols) : load_cols<T>(weight, column(i), a.cols);

    RowVecs<T, SHIFT, VEC == 8 && !QUANT> in{a.cols, 0};
    in.init(sh, nvec, t, tpr);
    int s = 0;
    uint32_t phase = 0;
    for (long long r = blockIdx.x; r < a.rows; r += step) {
        const long long off = r * a.cols;
        if (!mbar_wait_bounded(smem_u32(bars + s), phase, kRowWaitNs)) {
            give_up(smem_u32(bars), s, phase, slots, err);
            return;
        }
        const unsigned char *slot = ring + s * slot_bytes;
        in.at(r, total);
        float y[NV][VEC];
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = column(i);
            unpack16<T>(in.load(slot, a.x, i, c), y[i]);
            if (a.residual) {
                float g[VEC];
                unpack16<T>(in.load(slot + row_bytes, a.residual, i, c), g);
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[i][j] += g[j];
                const uint4 h = pack16<T>(y[i]);
                store_vec<T, SHIFT>(static_cast<T *>(a.residual_out) + off, c, a.cols, h);
                unpack16<T>(h, y[i]);
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) ss = fmaf(y[i][j], y[i][j], ss);
        }
        ss = team_reduce<SumOp, 0>(ss, red, turn);  // behind its barrier the slot has been read
        if (t == 0) stage(r + slots * step, s);
        if (++s == slots) {
            s = 0;
            phase ^= 1;
        }
        const float rstd = 1.0f / sqrtf(ss / (float)a.cols + a.eps);
        if (a.rstd && t == 0) a.rstd[r] = rstd;
        float gmax[NV], before[NV], amax = 0.0f;
        const int lo = a.group && t % GL == 0 ? sh : 0;  // tpr is a multiple of GL: the same for all vectors
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = column(i);
            if (weight) {
                float g[VEC];
                unpack16<T>(w[i], g);
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[i][j] = y[i][j] * rstd * g[j];
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[i][j] *= rstd;
            }
            if (!QUANT || a.out) store_vec<T, SHIFT>(static_cast<T *>(a.out) + off, c, a.cols, pack16<T>(y[i]));
            if (QUANT) {
                gmax[i] = vec_max<VEC, SHIFT>(y[i], lo, before[i]);
                amax = max_nan(amax, gmax[i]);
            }
        }
        if constexpr (QUANT) {
            Scale s8 = {}, s0 = {};
            if (!a.group) {
                s8 = with_inverse(scale_of(team_reduce<MaxOp, 0>(amax, red, turn), a.quant));
                if (t == 0) a.scale[r] = s8.s;
            } else if (SHIFT) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int v = t + i * tpr;
                    const float m = lanes_reduce<MaxOp, (GL < 32 ? GL : 32)>(gmax[i]);
                    if (v % GL == 0 && v * VEC < a.cols) atomicMax(&gmax_s[v / GL], __float_as_int(m));
                    if (lo && v && column(i) < a.cols) atomicMax(&gmax_s[v / GL - 1], __float_as_int(before[i]));
                }
                __syncthreads();
                for (int i = t; i < a.groups; i += tpr) {
                    const float sc = scale_of(__int_as_float(gmax_s[i]), a.quant);
                    a.scale[r * a.groups + i] = sc;
                    scale_s[i] = with_inverse(sc);
                    gmax_s[i] = 0;
                }
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = t + i * tpr, c = column(i);
                if (a.group && !SHIFT) {
                    s8 = with_inverse(scale_of(lanes_reduce<MaxOp, (GL < 32 ? GL : 32)>(gmax[i]), a.quant));
                    if (v % GL == 0 && c < a.cols) a.scale[r * a.groups + c / 128] = s8.s;
                } else if (a.group) {
                    // a vector behind the start of a group that is not there only holds the end of the last one
                    s8 = scale_s[min(v / GL, a.groups - 1)];
                    if (lo && v && c < a.cols) s0 = scale_s[v / GL - 1];
                }
                store_codes<VEC, SHIFT>(static_cast<unsigned char *>(a.out8) + off, c, a.cols, y[i], s8, s0, lo, a.quant);
            }
        }
    }
}

// Tensors out of step with one another, by elements; warp or CTA teams of C columns a thread.
template <typename T, int TPR, int C, bool QUANT>
__global__ void __launch_bounds__(TPR == 0 ? 1024 : kTeamThreads, TPR == 0 ? 1 : ctas_per_sm(C))
    norm_forward_elems_kernel(const NormArgs a) {
    __shared__ float red[64];
    // maxima of the groups (bits of values >= 0, two rows' sets), the scales that follow from them and their inverses
    __shared__ int gmax_s[2][TPR == 0 && QUANT ? 128 : 1];
    __shared__ Scale scale_s[TPR == 0 && QUANT ? 128 : 1];
    const int tpr = TPR == 0 ? (int)blockDim.x : TPR;
    const int t = TPR == 0 ? (int)threadIdx.x : (int)threadIdx.x % 32;
    const int teams = TPR == 0 ? 1 : kTeamThreads / 32, team = TPR == 0 ? 0 : (int)threadIdx.x / 32;
    int turn = 0, set = 0;
    float w[C];
    if (a.weight) load_elems<T, C>(static_cast<const T *>(a.weight), t, tpr, a.cols, w);
    if (TPR == 0 && QUANT) {
        for (int i = t; i < 256; i += tpr) gmax_s[i / 128][i % 128] = 0;
        __syncthreads();
    }
    const long long step = (long long)gridDim.x * teams;
    for (long long r = (long long)blockIdx.x * teams + team; r < a.rows; r += step) {  // the same in the whole team
        const long long off = r * a.cols;
        float y[C], ss = 0.0f;
        load_elems<T, C>(static_cast<const T *>(a.x) + off, t, tpr, a.cols, y);
        if (a.residual) {
            float g[C];
            load_elems<T, C>(static_cast<const T *>(a.residual) + off, t, tpr, a.cols, g);
            T *dst = static_cast<T *>(a.residual_out) + off;
#pragma unroll
            for (int k = 0; k < C; ++k) {
                const T h = from_f32<T>(y[k] + g[k]);
                if (k * tpr + t < a.cols) dst[k * tpr + t] = h;
                y[k] = to_f32(h);
            }
        }
#pragma unroll
        for (int k = 0; k < C; ++k) ss = fmaf(y[k], y[k], ss);
        ss = team_reduce<SumOp, TPR>(ss, red, turn);
        const float rstd = 1.0f / sqrtf(ss / (float)a.cols + a.eps);
        if (a.rstd && t == 0) a.rstd[r] = rstd;
        float amax = 0.0f;
#pragma unroll
        for (int k = 0; k < C; ++k) {
            y[k] *= rstd;
            if (a.weight) y[k] *= w[k];
            const bool in = k * tpr + t < a.cols;
            if (in && (!QUANT || a.out)) static_cast<T *>(a.out)[off + k * tpr + t] = from_f32<T>(y[k]);
            if (QUANT) {
                if (!in) y[k] = 0.0f;
                amax = max_nan(amax, fabsf(y[k]));
            }
        }
        if constexpr (QUANT) {
            Scale s = {};
            if (!a.group) {
                s = with_inverse(scale_of(team_reduce<MaxOp, TPR>(amax, red, turn), a.quant));
                if (t == 0) a.scale[r] = s.s;
            } else if (TPR == 0) {
                // 32 columns of a warp lie in one group
#pragma unroll
                for (int k = 0; k < C; ++k) {
                    const float m = lanes_reduce<MaxOp, 32>(fabsf(y[k]));
                    const int c = k * tpr + t - t % 32;
                    if (t % 32 == 0 && c < a.cols) atomicMax(&gmax_s[set][c / 128], __float_as_int(m));
                }
                __syncthreads();
                for (int i = t; i < a.groups; i += tpr) {
                    s = with_inverse(scale_of(__int_as_float(gmax_s[set][i]), a.quant));
                    scale_s[i] = s;
                    a.scale[r * a.groups + i] = s.s;
                    gmax_s[set ^ 1][i] = 0;  // the next row's, last read two barriers ago
                }
                __syncthreads();
                set ^= 1;
            }
            unsigned char *dst = static_cast<unsigned char *>(a.out8) + off;
#pragma unroll
            for (int k = 0; k < C; ++k) {
                const int c = k * tpr + t;
                if (a.group && TPR == 0) {
                    s = scale_s[c < a.cols ? c / 128 : 0];
                } else if (a.group && k % 4 == 0) {
                    // a warp's values k .. k + 3 are 128 columns
                    float m = fabsf(y[k]);
#pragma unroll
                    for (int q = 1; q < 4; ++q)
                        if (k + q < C) m = max_nan(m, fabsf(y[k + q]));
                    s = with_inverse(scale_of(lanes_reduce<MaxOp, 32>(m), a.quant));
                    if (t == 0 && c < a.cols) a.scale[r * a.groups + k / 4] = s.s;
                }
                if (c < a.cols) {
                    dst[c] = code_of(y[k], s, a.quant);
                }
            }
        }
    }
}

template <typename T, int TPR, int C>
cudaError_t launch_elems(const NormArgs &a, int threads, const DeviceInfo *dev, cudaStream_t stream) {
    const int teams = TPR == 0 ? 1 : threads / 32;
    const long long need = (a.rows + teams - 1) / teams;
    const long long most = (long long)dev->sms * (TPR == 0 ? 1024 / threads : ctas_per_sm(C));
    const unsigned grid = (unsigned)(need < most ? need : most);
    if (a.quant) norm_forward_elems_kernel<T, TPR, C, true><<<grid, threads, 0, stream>>>(a);
    else norm_forward_elems_kernel<T, TPR, C, false><<<grid, threads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, int TPR, int NV, bool SHIFT>
cudaError_t launch_one(const NormArgs &a, const DeviceInfo *dev, cudaStream_t stream) {
    constexpr int teams = kTeamThreads / TPR;
    const long long need = (a.rows + teams - 1) / teams, most = (long long)dev->sms * ctas_per_sm(NV * Storage<T>::kVec);
    const unsigned grid = (unsigned)(need < most ? need : most);
    if (a.quant) norm_forward_kernel<T, TPR, NV, true, SHIFT><<<grid, kTeamThreads, 0, stream>>>(a);
    else norm_forward_kernel<T, TPR, NV, false, SHIFT><<<grid, kTeamThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, bool SHIFT> cudaError_t launch_wide(const NormArgs &a, const DeviceInfo *dev, cudaStream_t stream) {
    constexpr int VEC = Storage<T>::kVec;
    const int span = a.cols + (SHIFT ? VEC - 1 : 0), threads = ((span + 15) / 16 + 31) / 32 * 32;  // at most 1024
    const int slot = (span + VEC - 1) / VEC * 16 * (a.residual ? 2 : 1);
    // as many CTAs as the registers allow (64 a thread), fewer where a slot would not fit their share
    int per_sm = 1024 / threads;
    if (per_sm > 8) per_sm = 8;
    while (per_sm > 1 && 2 * slot > staged_budget(per_sm)) --per_sm;
    int slots = staged_budget(per_sm) / slot;
    if (slots > 4) slots = 4;
    const int smem = slots * slot;
    static std::atomic<bool> plain_ok[kMaxDev], quant_ok[kMaxDev];
    const cudaError_t e = a.quant ? allow_smem(norm_forward_wide_kernel<T, true, SHIFT>, staged_budget(1), quant_ok)
                                  : allow_smem(norm_forward_wide_kernel<T, false, SHIFT>, staged_budget(1), plain_ok);
    if (e != cudaSuccess) return e;
    long long most = (long long)dev->sms * per_sm;
    if (SHIFT) most -= most % VEC;  // a CTA's rows have the same shift
    const unsigned grid = (unsigned)(a.rows < most ? a.rows : most);
    if (a.quant) norm_forward_wide_kernel<T, true, SHIFT><<<grid, threads, smem, stream>>>(a, slots, dev->err);
    else norm_forward_wide_kernel<T, false, SHIFT><<<grid, threads, smem, stream>>>(a, slots, dev->err);
    return cudaGetLastError();
}

template <typename T, bool SHIFT> cudaError_t launch_vec(const NormArgs &a, const DeviceInfo *dev, cudaStream_t stream) {
    constexpr int VEC = Storage<T>::kVec;
    const int nvec = (a.cols + (SHIFT ? VEC - 1 : 0) + VEC - 1) / VEC;
    if (nvec <= 8) return launch_one<T, 8, 1, SHIFT>(a, dev, stream);
    if (nvec <= 16) return launch_one<T, 16, 1, SHIFT>(a, dev, stream);
    if (nvec <= 32) return launch_one<T, 32, 1, SHIFT>(a, dev, stream);
    if (nvec <= 64) return launch_one<T, 32, 2, SHIFT>(a, dev, stream);
    if (nvec <= 128) return launch_one<T, 32, 4, SHIFT>(a, dev, stream);
    return launch_wide<T, SHIFT>(a, dev, stream);
}

template <typename T> cudaError_t launch_t(const NormArgs &a, cudaStream_t stream) {
    constexpr int VEC = Storage<T>::kVec;
    const DeviceInfo *dev = device_info();
    if (!dev) return cudaErrorNotSupported;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.x), res = reinterpret_cast<uintptr_t>(a.residual);
    const uintptr_t res_out = reinterpret_cast<uintptr_t>(a.residual_out), out = reinterpret_cast<uintptr_t>(a.out);
    const uintptr_t out8 = reinterpret_cast<uintptr_t>(a.out8);
    const uintptr_t bits = x | res | reinterpret_cast<uintptr_t>(a.weight) | res_out | out | out8 |
                           (uintptr_t)((size_t)a.cols * sizeof(T));
    if (bits % 16 == 0) return launch_vec<T, false>(a, dev, stream);
    // in step: an element of all tensors is equally far from a vector's start
    const bool in_step = (!res || ((x ^ res) % 16 == 0 && (x ^ res_out) % 16 == 0)) && (!out || (x ^ out) % 16 == 0) &&
                         (!out8 || out8 % VEC == x % 16 / sizeof(T));
    // four vectors a lane of shifted fp32 lose to elements: 40000 x 301 38.3 us against 32.7 (e4m3 44.7 against 36.6),
    // 20011 x 501 29.3 against 28.4; narrower and wider rows, and 16 bits, gain: fp16 5734 x 4383 42 us against 72 (e4m3
    // 51 against 127), 100000 x 61 fp32 20 against 25
    const int nvec = (a.cols + 2 * (VEC - 1)) / VEC;
    if (in_step && a.cols + VEC - 1 <= 16384 && !(VEC == 4 && nvec > 64 && nvec <= 128))
        return launch_vec<T, true>(a, dev, stream);
    if (a.cols <= 128) return launch_elems<T, 32, 4>(a, kTeamThreads, dev, stream);
    if (a.cols <= 512) return launch_elems<T, 32, 16>(a, kTeamThreads, dev, stream);
    return launch_elems<T, 0, 16>(a, ((a.cols + 15) / 16 + 31) / 32 * 32, dev, stream);  // at most 1024 threads
}

}  // namespace

cudaError_t launch_norm_forward(const NormArgs &a, cudaStream_t stream) {
    switch (a.dtype) {
        case DType::F32: return launch_t<float>(a, stream);
        case DType::F16: return launch_t<__half>(a, stream);
        case DType::BF16: return launch_t<__nv_bfloat16>(a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace dcnb
