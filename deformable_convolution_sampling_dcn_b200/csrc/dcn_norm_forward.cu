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
#include "dcn_launch.h"
#include "dcn_norm.cuh"

namespace dcnb {
namespace {

constexpr float kScaleMin = 1.17549435e-38f;  // 2^-126: 1 / s stays finite, an all-zero row gives q = 0

// Four values to four 8-bit codes, in memory order.  A NaN becomes the e4m3
// NaN, and 0 in int8 (its scale is NaN).
__device__ __forceinline__ uint32_t pack8(const float *y, float inv, int quant) {
    if (quant == kQuantE4M3) {
        const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0] * inv, y[1] * inv), __NV_SATFINITE,
                                                                 __NV_E4M3);
        const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2] * inv, y[3] * inv), __NV_SATFINITE,
                                                                 __NV_E4M3);
        return (uint32_t)lo | ((uint32_t)hi << 16);
    }
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int q = max(-127, min(127, __float2int_rn(y[i] * inv)));
        w |= (uint32_t)(q & 255) << (8 * i);
    }
    return w;
}

template <typename T, int TPR, int NV, bool AL>
__global__ void __launch_bounds__(TPR == 0 ? 1024 : 256) norm_forward_kernel(const NormArgs a) {
    constexpr int VEC = Storage<T>::kVec;
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

    const long long step = (long long)gridDim.x * teams;
    // every lane of a warp runs the same number of rounds: the shuffles need them all
    for (long long base = (long long)blockIdx.x * teams; base < a.rows; base += step) {
        const long long r = base + team;
        const bool live = r < a.rows;
        const long long off = live ? r * a.cols : 0;
        const int cols = live ? a.cols : 0;
        uint4 hv[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) hv[i] = load_cols<T, AL>(x + off, (t + i * tpr) * VEC, cols);
        if (res) {
            uint4 rv[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) rv[i] = load_cols<T, AL>(res + off, (t + i * tpr) * VEC, cols);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float f[VEC], g[VEC];
                unpack16<T>(hv[i], f);
                unpack16<T>(rv[i], g);
#pragma unroll
                for (int j = 0; j < VEC; ++j) f[j] += g[j];
                hv[i] = pack16<T>(f);
                store_cols<T, AL>(static_cast<T *>(a.residual_out) + off, (t + i * tpr) * VEC, cols, hv[i]);
            }
        }
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[VEC];
            unpack16<T>(hv[i], f);
#pragma unroll
            for (int j = 0; j < VEC; ++j) ss = fmaf(f[j], f[j], ss);
        }
        ss = team_reduce<SumOp, TPR>(ss, red, turn);
        const float rstd = 1.0f / sqrtf(ss / (float)a.cols + a.eps);
        if (a.rstd && t == 0 && live) a.rstd[r] = rstd;

        float amax = 0.0f;
        float gmax[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[VEC];
            unpack16<T>(hv[i], f);
            if (weight) {
                float g[VEC];
                unpack16<T>(w[i], g);
#pragma unroll
                for (int j = 0; j < VEC; ++j) f[j] = f[j] * rstd * g[j];
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) f[j] *= rstd;
            }
            if (a.out) store_cols<T, AL>(static_cast<T *>(a.out) + off, (t + i * tpr) * VEC, cols, pack16<T>(f));
            if (a.quant) {
                gmax[i] = 0.0f;
                if (AL || (t + i * tpr) * VEC < cols) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const bool in = AL || (t + i * tpr) * VEC + j < cols;
                        gmax[i] = max_nan(gmax[i], in ? fabsf(f[j]) : 0.0f);
                    }
                }
                amax = max_nan(amax, gmax[i]);
            }
        }
        if (!a.quant) continue;

        const float top = a.quant == kQuantE4M3 ? 448.0f : 127.0f;
        // lanes that share 128 columns; a team narrower than that holds rows of at most 128 columns
        constexpr int GL = 128 / VEC;
        const bool grouped = a.group != 0 && (TPR == 0 || TPR >= GL);
        float s_row = 0.0f;
        if (!grouped) {
            s_row = max_nan(team_reduce<MaxOp, TPR>(amax, red, turn) / top, kScaleMin);
            if (t == 0 && live) a.scale[r] = s_row;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = t + i * tpr, c = v * VEC;
            float s = s_row;
            if (grouped) {
                s = max_nan(lanes_reduce<MaxOp, (GL < 32 ? GL : 32)>(gmax[i]) / top, kScaleMin);
                if (v % GL == 0 && c < cols) a.scale[r * a.groups + c / 128] = s;
            }
            if (c < cols) {
                const float inv = 1.0f / s;
                float f[VEC];
                unpack16<T>(hv[i], f);
                if (weight) {
                    float g[VEC];
                    unpack16<T>(w[i], g);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) f[j] = f[j] * rstd * g[j];
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) f[j] *= rstd;
                }
                uint32_t q[VEC / 4];
#pragma unroll
                for (int j = 0; j < VEC / 4; ++j) q[j] = pack8(f + 4 * j, inv, a.quant);
                unsigned char *dst = static_cast<unsigned char *>(a.out8) + off + c;
                if constexpr (AL) {
                    if constexpr (VEC == 8)
                        *reinterpret_cast<uint2 *>(dst) = make_uint2(q[0], q[1]);
                    else
                        *reinterpret_cast<uint32_t *>(dst) = q[0];
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j)
                        if (c + j < cols) dst[j] = (unsigned char)(q[j / 4] >> (8 * (j % 4)));
                }
            }
        }
    }
}

template <typename T, int TPR, int NV, bool AL>
cudaError_t launch_one(const NormArgs &a, int threads, const DeviceInfo *dev, cudaStream_t stream) {
    const int teams = TPR == 0 ? 1 : threads / TPR;
    const long long need = (a.rows + teams - 1) / teams;
    // 2048 threads an SM (the kernels stay below 64 registers, at 32 and fewer they all fit)
    const long long most = (long long)dev->sms * (2048 / threads);
    norm_forward_kernel<T, TPR, NV, AL><<<(unsigned)(need < most ? need : most), threads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, bool AL> cudaError_t launch_al(const NormArgs &a, cudaStream_t stream) {
    const DeviceInfo *dev = device_info();
    if (!dev) return cudaErrorNotSupported;
    constexpr int VEC = Storage<T>::kVec;
    const int nvec = (a.cols + VEC - 1) / VEC;
    if (nvec <= 8) return launch_one<T, 8, 1, AL>(a, 256, dev, stream);
    if (nvec <= 32) return launch_one<T, 32, 1, AL>(a, 256, dev, stream);
    if (nvec <= 64) return launch_one<T, 32, 2, AL>(a, 256, dev, stream);
    if (nvec <= 128) return launch_one<T, 32, 4, AL>(a, 256, dev, stream);
    const int threads = ((nvec + 3) / 4 + 31) / 32 * 32;  // at most 1024: cols <= 16384
    return launch_one<T, 0, 4, AL>(a, threads, dev, stream);
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
