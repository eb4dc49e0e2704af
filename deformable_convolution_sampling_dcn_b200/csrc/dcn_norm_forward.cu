// Residual addition and root-mean-square norm, with the output in the storage
// type, in 8 bits with scales, or both:
//   h    = rnd(x + residual)             (h = x without a residual)
//   rstd = 1 / sqrt(mean_c(h^2) + eps)
//   y    = h * rstd * weight
//   8 bit: s = max(max|y| / top, 2^-126) over the row or over 128 columns,
//          q = rnd(y * (1 / s)), top = 448 (e4m3) or 127 (int8)
// h is rounded to the storage type first because that is the value the next
// block's residual and the backward pass read; everything after it is fp32 and
// rounded once.
//
// Bound: device memory.  One pass: a row stays in the registers of its team
// between the statistics and the output, so each byte moves once.
#include <cuda_fp8.h>

#include "dcn_device.h"
#include "dcn_host.h"
#include "dcn_launch.h"
#include "dcn_norm.cuh"

namespace dcnb {
namespace {

constexpr float kScaleMin = 1.17549435e-38f;  // 2^-126: 1 / s stays finite, an all-zero row gives q = 0

// Four values to four 8-bit codes, in memory order.  int8 rounds by adding
// 1.5 * 2^23 in the fused product: the low byte of the sum is the rounded value
// (|y * inv| <= 127 * (1 + 2^-22)).
__device__ __forceinline__ uint32_t pack8(const float *y, float inv, int quant) {
    if (quant == kQuantE4M3) {
        const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0] * inv, y[1] * inv), __NV_SATFINITE,
                                                                 __NV_E4M3);
        const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2] * inv, y[3] * inv), __NV_SATFINITE,
                                                                 __NV_E4M3);
        return (uint32_t)lo | ((uint32_t)hi << 16);
    }
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = __float_as_uint(fmaf(y[i], inv, 12582912.0f));
    return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
}

// The codes of a thread's vector at an address that is a multiple of VEC.
template <int VEC>
__device__ __forceinline__ void store_codes(unsigned char *dst, const float *y, float inv, int quant) {
    if constexpr (VEC == 8)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack8(y, inv, quant), pack8(y + 4, inv, quant));
    else
        *reinterpret_cast<uint32_t *>(dst) = pack8(y, inv, quant);
}

constexpr int kMaxSlots = 8;

// A thread holds C = NV * VEC columns of a row: up to 16 with the loads of its
// team's next row in flight meanwhile, or 32 without.  8-lane and warp teams
// share a CTA of 256 threads, a CTA team has up to 512; CTAs on an SM follow
// from the registers that leaves (48, 80 or 128).
constexpr int kTeamThreads = 256;
template <int TPR> constexpr int max_threads() { return TPR == 0 ? 512 : kTeamThreads; }
constexpr int threads_per_sm(int c) { return c <= 8 ? 1280 : c <= 16 ? 768 : 512; }

template <typename T, int TPR, int NV, bool AL, bool QUANT>
__global__ void __launch_bounds__(max_threads<TPR>(), threads_per_sm(NV * Storage<T>::kVec) / max_threads<TPR>())
    norm_forward_kernel(const NormArgs a) {
    constexpr int VEC = Storage<T>::kVec;
    constexpr bool AHEAD = NV * VEC <= 16;
    __shared__ float red[64];
    const int tpr = TPR == 0 ? (int)blockDim.x : TPR;
    const int t = TPR == 0 ? (int)threadIdx.x : (int)threadIdx.x % TPR;
    const int teams = TPR == 0 ? 1 : (int)blockDim.x / TPR;
    const int team = TPR == 0 ? 0 : (int)threadIdx.x / TPR;
    int turn = 0;
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    const T *weight = static_cast<const T *>(a.weight);
    uint4 w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (weight) w[i] = load_cols<T, AL>(weight, (t + i * tpr) * VEC, a.cols);

    uint4 xn[NV], rn[NV];
    auto fetch = [&](long long r) {
        const long long off = r < a.rows ? r * a.cols : 0;
        const int cols = r < a.rows ? a.cols : 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            xn[i] = load_cols<T, AL>(x + off, (t + i * tpr) * VEC, cols);
            if (res) rn[i] = load_cols<T, AL>(res + off, (t + i * tpr) * VEC, cols);
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
            unpack16<T>(xn[i], y[i]);
            if (res) {
                float g[VEC];
                unpack16<T>(rn[i], g);
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[i][j] += g[j];
                const uint4 h = pack16<T>(y[i]);
                store_cols<T, AL>(static_cast<T *>(a.residual_out) + off, (t + i * tpr) * VEC, cols, h);
                unpack16<T>(h, y[i]);
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) ss = fmaf(y[i][j], y[i][j], ss);
        }
        if (AHEAD) fetch(r + step);
        ss = team_reduce<SumOp, TPR>(ss, red, turn);
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
                store_cols<T, AL>(static_cast<T *>(a.out) + off, (t + i * tpr) * VEC, cols, pack16<T>(y[i]));
        }
        if constexpr (QUANT) {
            float amax = 0.0f, gmax[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                gmax[i] = 0.0f;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    // columns past the row hold 0 * rstd * 0, which is NaN where rstd is
                    const bool in = (t + i * tpr) * VEC + (AL ? 0 : j) < cols;
                    gmax[i] = max_nan(gmax[i], in ? fabsf(y[i][j]) : 0.0f);
                }
                amax = max_nan(amax, gmax[i]);
            }
            const float top = a.quant == kQuantE4M3 ? 448.0f : 127.0f;
            // lanes that share 128 columns; a team narrower than that holds rows of at most 128 columns
            constexpr int GL = 128 / VEC;
            const bool grouped = a.group != 0 && (TPR == 0 || TPR >= GL);
            float s = 0.0f, inv = 0.0f;
            if (!grouped) {
                s = max_nan(team_reduce<MaxOp, TPR>(amax, red, turn) / top, kScaleMin);
                inv = 1.0f / s;
                if (t == 0 && live) a.scale[r] = s;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = t + i * tpr, c = v * VEC;
                if (grouped) {
                    s = max_nan(lanes_reduce<MaxOp, (GL < 32 ? GL : 32)>(gmax[i]) / top, kScaleMin);
                    inv = 1.0f / s;
                    if (v % GL == 0 && c < cols) a.scale[r * a.groups + c / 128] = s;
                }
                if (c < cols) {
                    unsigned char *dst = static_cast<unsigned char *>(a.out8) + off + c;
                    if constexpr (AL) {
                        store_codes<VEC>(dst, y[i], inv, a.quant);
                    } else {
                        uint32_t q[VEC / 4];
#pragma unroll
                        for (int j = 0; j < VEC / 4; ++j) q[j] = pack8(y[i] + 4 * j, inv, a.quant);
#pragma unroll
                        for (int j = 0; j < VEC; ++j)
                            if (c + j < cols) dst[j] = (unsigned char)(q[j / 4] >> (8 * (j % 4)));
                    }
                }
            }
        }
    }
}

// Rows wider than a warp team holds, 16-byte aligned: a CTA of 16 columns a
// thread per row, the rows staged by bulk copies (bf16 2047 x 4096 to int8: 16.8
// us with the next row's loads in registers, 13.8 us staged).
template <typename T, bool QUANT>
__global__ void __launch_bounds__(1024, 1) norm_forward_wide_kernel(const NormArgs a, int slots, unsigned int *err) {
    constexpr int VEC = Storage<T>::kVec, NV = 16 / VEC, GL = 128 / VEC;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ float red[64];
    __shared__ __align__(8) uint64_t bars[kMaxSlots];
    const int t = threadIdx.x, tpr = blockDim.x;
    const uint32_t row_bytes = (uint32_t)a.cols * sizeof(T), slot_bytes = a.residual ? 2 * row_bytes : row_bytes;
    const T *weight = static_cast<const T *>(a.weight);
    int turn = 0;
    if (t == 0) {
        for (int i = 0; i < slots; ++i) mbar_init(smem_u32(bars + i), 1);
        fence_mbar_init();
    }
    __syncthreads();
    auto stage = [&](long long r, int s) {  // by thread 0
        if (r >= a.rows) return;
        const uint32_t bar = smem_u32(bars + s), dst = smem_u32(ring) + s * slot_bytes;
        mbar_arrive_expect_tx(bar, slot_bytes);
        bulk_load(dst, static_cast<const T *>(a.x) + r * a.cols, row_bytes, bar);
        if (a.residual) bulk_load(dst + row_bytes, static_cast<const T *>(a.residual) + r * a.cols, row_bytes, bar);
    };
    const long long step = gridDim.x;
    if (t == 0)
        for (int i = 0; i < slots; ++i) stage(blockIdx.x + i * step, i);
    uint4 w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (weight) w[i] = load_cols<T, true>(weight, (t + i * tpr) * VEC, a.cols);

    int s = 0;
    uint32_t phase = 0;
    for (long long r = blockIdx.x; r < a.rows; r += step) {
        const long long off = r * a.cols;
        if (!mbar_wait_bounded(smem_u32(bars + s), phase, kRowWaitNs)) {
            give_up(smem_u32(bars), s, phase, slots, err);
            return;
        }
        const unsigned char *slot = ring + s * slot_bytes;
        float y[NV][VEC];
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * tpr) * VEC;
            unpack16<T>(load_cols<T, true>(reinterpret_cast<const T *>(slot), c, a.cols), y[i]);
            if (a.residual) {
                float g[VEC];
                unpack16<T>(load_cols<T, true>(reinterpret_cast<const T *>(slot + row_bytes), c, a.cols), g);
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[i][j] += g[j];
                const uint4 h = pack16<T>(y[i]);
                store_cols<T, true>(static_cast<T *>(a.residual_out) + off, c, a.cols, h);
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
        float gmax[NV], amax = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * tpr) * VEC;
            if (weight) {
                float g[VEC];
                unpack16<T>(w[i], g);
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[i][j] = y[i][j] * rstd * g[j];
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[i][j] *= rstd;
            }
            if (!QUANT || a.out) store_cols<T, true>(static_cast<T *>(a.out) + off, c, a.cols, pack16<T>(y[i]));
            if (QUANT) {
                gmax[i] = 0.0f;
                if (c < a.cols) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) gmax[i] = max_nan(gmax[i], fabsf(y[i][j]));
                }
                amax = max_nan(amax, gmax[i]);
            }
        }
        if constexpr (QUANT) {
            const float top = a.quant == kQuantE4M3 ? 448.0f : 127.0f;
            float sc = 0.0f, inv = 0.0f;
            if (!a.group) {
                sc = max_nan(team_reduce<MaxOp, 0>(amax, red, turn) / top, kScaleMin);
                inv = 1.0f / sc;
                if (t == 0) a.scale[r] = sc;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = t + i * tpr, c = v * VEC;
                if (a.group) {
                    sc = max_nan(lanes_reduce<MaxOp, (GL < 32 ? GL : 32)>(gmax[i]) / top, kScaleMin);
                    inv = 1.0f / sc;
                    if (v % GL == 0 && c < a.cols) a.scale[r * a.groups + c / 128] = sc;
                }
                if (c < a.cols) store_codes<VEC>(static_cast<unsigned char *>(a.out8) + off + c, y[i], inv, a.quant);
            }
        }
    }
}

template <typename T, int TPR, int NV, bool AL>
cudaError_t launch_one(const NormArgs &a, int threads, const DeviceInfo *dev, cudaStream_t stream) {
    constexpr int VEC = Storage<T>::kVec;
    const int teams = TPR == 0 ? 1 : threads / TPR;
    const long long need = (a.rows + teams - 1) / teams;
    const long long most = (long long)dev->sms * (threads_per_sm(NV * VEC) / threads);
    const unsigned grid = (unsigned)(need < most ? need : most);
    if (a.quant) norm_forward_kernel<T, TPR, NV, AL, true><<<grid, threads, 0, stream>>>(a);
    else norm_forward_kernel<T, TPR, NV, AL, false><<<grid, threads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_wide(const NormArgs &a, const DeviceInfo *dev, cudaStream_t stream) {
    const int threads = ((a.cols + 15) / 16 + 31) / 32 * 32;  // at most 1024
    const int slot = a.cols * (int)sizeof(T) * (a.residual ? 2 : 1);
    // as many CTAs as the registers allow (64 a thread), fewer where a slot would not fit their share
    int per_sm = 1024 / threads;
    if (per_sm > 8) per_sm = 8;
    while (per_sm > 1 && 2 * slot > staged_budget(per_sm)) --per_sm;
    int slots = staged_budget(per_sm) / slot;
    if (slots > 4) slots = 4;
    const int smem = slots * slot;
    static std::atomic<bool> plain_ok[kMaxDev], quant_ok[kMaxDev];
    const cudaError_t e = a.quant ? allow_smem(norm_forward_wide_kernel<T, true>, staged_budget(1), quant_ok)
                                  : allow_smem(norm_forward_wide_kernel<T, false>, staged_budget(1), plain_ok);
    if (e != cudaSuccess) return e;
    const long long most = (long long)dev->sms * per_sm;
    const unsigned grid = (unsigned)(a.rows < most ? a.rows : most);
    if (a.quant) norm_forward_wide_kernel<T, true><<<grid, threads, smem, stream>>>(a, slots, dev->err);
    else norm_forward_wide_kernel<T, false><<<grid, threads, smem, stream>>>(a, slots, dev->err);
    return cudaGetLastError();
}

template <typename T, bool AL> cudaError_t launch_al(const NormArgs &a, cudaStream_t stream) {
    const DeviceInfo *dev = device_info();
    if (!dev) return cudaErrorNotSupported;
    constexpr int VEC = Storage<T>::kVec;
    const int nvec = (a.cols + VEC - 1) / VEC;
    if (nvec <= 8) return launch_one<T, 8, 1, AL>(a, kTeamThreads, dev, stream);
    if (nvec <= 32) return launch_one<T, 32, 1, AL>(a, kTeamThreads, dev, stream);
    if (nvec <= 64) return launch_one<T, 32, 2, AL>(a, kTeamThreads, dev, stream);
    if (nvec <= 128) return launch_one<T, 32, 4, AL>(a, kTeamThreads, dev, stream);
    if constexpr (AL) {
        return launch_wide<T>(a, dev, stream);
    } else {
        // at most 512 threads: 16 columns each up to 8192, 32 up to 16384
        const int nv = (a.cols <= 8192 ? 16 : 32) / VEC, threads = ((nvec + nv - 1) / nv + 31) / 32 * 32;
        if (nv == 16 / VEC) return launch_one<T, 0, 16 / VEC, AL>(a, threads, dev, stream);
        return launch_one<T, 0, 32 / VEC, AL>(a, threads, dev, stream);
    }
}

template <typename T> cudaError_t launch_t(const NormArgs &a, cudaStream_t stream) {
    uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual) |
                     reinterpret_cast<uintptr_t>(a.weight) | reinterpret_cast<uintptr_t>(a.residual_out) |
                     reinterpret_cast<uintptr_t>(a.out) | reinterpret_cast<uintptr_t>(a.out8) |
                     (uintptr_t)((size_t)a.cols * sizeof(T));
    return bits % 16 == 0 ? launch_al<T, true>(a, stream) : launch_al<T, false>(a, stream);
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
