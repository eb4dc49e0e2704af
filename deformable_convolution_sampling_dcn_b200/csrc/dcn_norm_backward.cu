// Gradients of the residual addition + root-mean-square norm
// (dcn_norm_forward.cu).  With xh = h * rstd and g = grad_out * weight,
//   grad_x      = rstd * (g - xh * mean_c(g * xh)) + grad_residual_out
//   grad_weight = sum_rows grad_out * xh
// grad_x is the gradient of x and of the residual alike (h is their sum).
//
// Bound: device memory.  The first kernel reads each row once, keeps it in its
// team's registers across the one reduction, and keeps the weight gradient of
// the columns it owns in fp32 registers over all of its rows; each CTA adds up
// its teams in shared memory and writes one row of partial sums.  The second
// kernel adds those rows in a fixed order, so the result does not depend on
// timing (no atomics).
#include "dcn_device.h"
#include "dcn_launch.h"
#include "dcn_norm.cuh"

namespace dcnb {
namespace {

template <typename T, int TPR, int NV, bool AL>
__global__ void __launch_bounds__(TPR == 0 ? 1024 : 256) norm_backward_kernel(const NormArgs a) {
    constexpr int VEC = Storage<T>::kVec;
    __shared__ float red[64];
    __shared__ float4 gws[TPR == 0 ? 1 : 256 * NV * VEC / 4];
    const int tpr = TPR == 0 ? (int)blockDim.x : TPR;
    const int t = TPR == 0 ? (int)threadIdx.x : (int)threadIdx.x % TPR;
    const int teams = TPR == 0 ? 1 : (int)blockDim.x / TPR;
    const int team = TPR == 0 ? 0 : (int)threadIdx.x / TPR;
    int turn = 0;
    const T *hp = static_cast<const T *>(a.h), *gyp = static_cast<const T *>(a.grad_out);
    const T *ghp = static_cast<const T *>(a.grad_residual_out), *weight = static_cast<const T *>(a.weight);
    uint4 w[NV];
    float gw[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (weight) w[i] = load_cols<T, AL>(weight, (t + i * tpr) * VEC, a.cols);
#pragma unroll
        for (int j = 0; j < VEC; ++j) gw[i][j] = 0.0f;
    }
    const float inv_cols = 1.0f / (float)a.cols;
    const long long step = (long long)gridDim.x * teams;
    for (long long base = (long long)blockIdx.x * teams; base < a.rows; base += step) {
        const long long r = base + team;
        const bool live = r < a.rows;
        const long long off = live ? r * a.cols : 0;
        const int cols = live ? a.cols : 0;
        const float rstd = live ? a.rstd[r] : 0.0f;
        uint4 hv[NV], gv[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            hv[i] = load_cols<T, AL>(hp + off, (t + i * tpr) * VEC, cols);
            gv[i] = load_cols<T, AL>(gyp + off, (t + i * tpr) * VEC, cols);
        }
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float h[VEC], gy[VEC], wf[VEC];
            unpack16<T>(hv[i], h);
            unpack16<T>(gv[i], gy);
            if (weight) unpack16<T>(w[i], wf);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float p = gy[j] * (h[j] * rstd);
                gw[i][j] += p;
                dot = weight ? fmaf(p, wf[j], dot) : dot + p;
            }
        }
        dot = team_reduce<SumOp, TPR>(dot, red, turn) * inv_cols;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float h[VEC], gy[VEC], wf[VEC], o[VEC];
            unpack16<T>(hv[i], h);
            unpack16<T>(gv[i], gy);
            if (weight) unpack16<T>(w[i], wf);
            uint4 rv = make_uint4(0, 0, 0, 0);
            if (ghp) rv = load_cols<T, AL>(ghp + off, (t + i * tpr) * VEC, cols);
            unpack16<T>(rv, o);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float g = weight ? gy[j] * wf[j] : gy[j];
                const float gx = rstd * (g - h[j] * rstd * dot);
                o[j] = ghp ? gx + o[j] : gx;
            }
            store_cols<T, AL>(static_cast<T *>(a.grad_x) + off, (t + i * tpr) * VEC, cols, pack16<T>(o));
        }
    }
    if (!a.grad_weight) return;
    float *part = a.partial + (long long)blockIdx.x * a.cols;
    if constexpr (TPR == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if ((t + i * tpr) * VEC + j < a.cols) part[(t + i * tpr) * VEC + j] = gw[i][j];
    } else {
        float *g = reinterpret_cast<float *>(gws);  // [teams][NV * TPR * VEC]
        constexpr int W = NV * TPR * VEC;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) g[team * W + (t + i * TPR) * VEC + j] = gw[i][j];
        __syncthreads();
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            float s = 0.0f;
            for (int k = 0; k < teams; ++k) s += g[k * W + c];
            part[c] = s;
        }
    }
}

// grad_weight[c] = sum over the CTAs of the first kernel, in a fixed order.
constexpr int kRedX = 32, kRedY = 16;
template <typename T>
__global__ void __launch_bounds__(kRedX *kRedY) norm_grad_weight_kernel(const float *partial, int n, int cols, T *out) {
    __shared__ float s[kRedY][kRedX];
    const int c = blockIdx.x * kRedX + threadIdx.x;
    float v = 0.0f;
    if (c < cols)
        for (int k = threadIdx.y; k < n; k += kRedY) v += partial[(long long)k * cols + c];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && c < cols) {
#pragma unroll
        for (int k = 1; k < kRedY; ++k) v += s[k][threadIdx.x];
        out[c] = from_f32<T>(v);
    }
}

template <typename T, int TPR, int NV, bool AL>
cudaError_t launch_one(const NormArgs &a, int threads, cudaStream_t stream) {
    const int teams = TPR == 0 ? 1 : threads / TPR;
    const long long need = (a.rows + teams - 1) / teams;
    const int grid = (int)(need < a.partial_rows ? need : a.partial_rows);
    norm_backward_kernel<T, TPR, NV, AL><<<grid, threads, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.grad_weight) return e;
    norm_grad_weight_kernel<T><<<(a.cols + kRedX - 1) / kRedX, dim3(kRedX, kRedY), 0, stream>>>(
        a.partial, grid, a.cols, static_cast<T *>(a.grad_weight));
    return cudaGetLastError();
}

template <typename T, bool AL> cudaError_t launch_al(const NormArgs &a, cudaStream_t stream) {
    constexpr int VEC = Storage<T>::kVec;
    constexpr int NVC = 16 / VEC;  // 2 or 4 vectors a thread in CTA teams: 16 columns
    const int nvec = (a.cols + VEC - 1) / VEC;
    if (nvec <= 8) return launch_one<T, 8, 1, AL>(a, 256, stream);
    if (nvec <= 32) return launch_one<T, 32, 1, AL>(a, 256, stream);
    if (nvec <= 64) return launch_one<T, 32, 2, AL>(a, 256, stream);
    const int threads = ((nvec + NVC - 1) / NVC + 31) / 32 * 32;  // at most 1024: cols <= 16384
    return launch_one<T, 0, NVC, AL>(a, threads, stream);
}

template <typename T> cudaError_t launch_t(const NormArgs &a, cudaStream_t stream) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.h) | reinterpret_cast<uintptr_t>(a.grad_out) |
                           reinterpret_cast<uintptr_t>(a.grad_residual_out) | reinterpret_cast<uintptr_t>(a.weight) |
                           reinterpret_cast<uintptr_t>(a.grad_x) | (uintptr_t)((size_t)a.cols * sizeof(T));
    return bits % 16 == 0 ? launch_al<T, true>(a, stream) : launch_al<T, false>(a, stream);
}

}  // namespace

int norm_backward_partial_rows(int64_t rows, int cols) {
    // four CTAs on each of 148 SMs: the partial rows do not depend on the device that asks for the size
    (void)cols;
    return (int)(rows < 592 ? rows : 592);
}

cudaError_t launch_norm_backward(const NormArgs &a, cudaStream_t stream) {
    switch (a.dtype) {
        case DType::F32: return launch_t<float>(a, stream);
        case DType::F16: return launch_t<__half>(a, stream);
        case DType::BF16: return launch_t<__nv_bfloat16>(a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace dcnb
