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

constexpr int kTeamThreads = 512;  // CTA of 8-lane and warp teams
constexpr int kSms = 148;

template <typename T, int TPR, int NV, bool AL>
__global__ void __launch_bounds__(TPR == 0 ? 1024 : kTeamThreads, TPR == 0 || NV * Storage<T>::kVec > 8 ? 1 : 2)
    norm_backward_kernel(const NormArgs a) {
    constexpr int VEC = Storage<T>::kVec;
    __shared__ float red[TPR == 0 ? 64 : 32 * NV * VEC];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
    // With one or two fp32 vectors a thread, the loads of a team's next row are in flight while it works on
    // the current one (bf16 102400 x 256: 46.1 -> 38.5 us); wider threads have no registers left for it
    // (fp32 12800 x 512: 29.5 us without, 32.5 us with, spilling).
    constexpr bool AHEAD = NV * VEC <= 8;
    uint4 hn[NV], gn[NV], rn[NV];
    float sn = 0.0f;
    auto fetch = [&](long long r) {
        const bool live = r < a.rows;
        const long long off = live ? r * a.cols : 0;
        const int cols = live ? a.cols : 0;
        sn = live ? a.rstd[r] : 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            hn[i] = load_cols<T, AL>(hp + off, (t + i * tpr) * VEC, cols);
            gn[i] = load_cols<T, AL>(gyp + off, (t + i * tpr) * VEC, cols);
            if (ghp) rn[i] = load_cols<T, AL>(ghp + off, (t + i * tpr) * VEC, cols);
        }
    };
    if (AHEAD) fetch((long long)blockIdx.x * teams + team);
    for (long long base = (long long)blockIdx.x * teams; base < a.rows; base += step) {
        const long long r = base + team;
        const bool live = r < a.rows;
        if (!AHEAD) fetch(r);
        uint4 hv[NV], gv[NV], rv[NV];
        const float rstd = sn;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            hv[i] = hn[i];
            gv[i] = gn[i];
            rv[i] = ghp ? rn[i] : make_uint4(0, 0, 0, 0);
        }
        if (AHEAD) fetch(r + step);
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
            unpack16<T>(rv[i], o);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float g = weight ? gy[j] * wf[j] : gy[j];
                const float gx = rstd * (g - h[j] * rstd * dot);
                o[j] = ghp ? gx + o[j] : gx;
            }
            store_cols<T, AL>(static_cast<T *>(a.grad_x) + (live ? r * a.cols : 0), (t + i * tpr) * VEC,
                              live ? a.cols : 0, pack16<T>(o));
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
        // one warp after the other adds its columns to the CTA's sums; 8-lane teams of a warp first
        // among themselves
        constexpr int W = TPR * NV * VEC;
        for (int k = 0; k < kTeamThreads / 32; ++k) {
            if ((int)threadIdx.x / 32 == k) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        float v = gw[i][j];
                        if (TPR == 8) {
                            v += __shfl_xor_sync(0xffffffffu, v, 8);
                            v += __shfl_xor_sync(0xffffffffu, v, 16);
                        }
                        // lane-major, so neighbouring lanes use neighbouring banks
                        float *s = red + (i * VEC + j) * TPR + t;
                        if (TPR == 32 || (threadIdx.x & 31) < TPR) *s = k ? *s + v : v;
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < W && c < a.cols; c += kTeamThreads) {
            const int v = c / VEC;
            part[c] = red[(v / TPR * VEC + c % VEC) * TPR + v % TPR];
        }
    }
}

// grad_weight[c] = sum over the CTAs of the first kernel, in a fixed order.  8
// columns (one 32-byte sector of a row of partial sums) and 128 threads along
// the rows: a few loads per thread, all in flight at once.
constexpr int kRedX = 8, kRedY = 128;
template <typename T>
__global__ void __launch_bounds__(kRedX *kRedY) norm_grad_weight_kernel(const float *partial, int n, int cols, T *out) {
    __shared__ float s[kRedY][kRedX];
    const int x = threadIdx.x % kRedX, y = threadIdx.x / kRedX, c = blockIdx.x * kRedX + x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float v = 0.0f;
    if (c < cols) {
#pragma unroll 4
        for (int k = y; k < n; k += kRedY) v += __ldcg(partial + (long long)k * cols + c);
    }
    s[y][x] = v;
    __syncthreads();
#pragma unroll
    for (int h = kRedY / 2; h > 0; h >>= 1) {
        if (y < h) s[y][x] += s[y + h][x];
        __syncthreads();
    }
    if (y == 0 && c < cols) out[c] = from_f32<T>(s[0][x]);
}

// Team, CTA size and CTAs on an SM for a row of nvec vectors (16-byte vectors
// of 4 or 8 columns).  A warp holds up to 128 vectors in registers; wider rows
// take a CTA with 16 columns a thread.
struct Config {
    int tpr, nv, threads, per_sm;
};
Config config_of(int cols, int vec) {
    const int nvec = (cols + vec - 1) / vec;
    if (nvec <= 8) return {8, 1, kTeamThreads, 2};
    if (nvec <= 32) return {32, 1, kTeamThreads, 2};
    if (nvec <= 64) return {32, 2, kTeamThreads, vec == 4 ? 2 : 1};
    if (nvec <= 128) return {32, 4, kTeamThreads, 1};
    const int nv = 16 / vec, threads = ((nvec + nv - 1) / nv + 31) / 32 * 32;  // at most 1024: cols <= 16384
    const int fit = 1024 / threads;
    return {0, nv, threads, fit < 8 ? fit : 8};
}

template <typename T, int TPR, int NV, bool AL>
cudaError_t launch_one(const NormArgs &a, int threads, cudaStream_t stream) {
    const int teams = TPR == 0 ? 1 : threads / TPR;
    const long long need = (a.rows + teams - 1) / teams;
    const int grid = (int)(need < a.partial_rows ? need : a.partial_rows);
    norm_backward_kernel<T, TPR, NV, AL><<<grid, threads, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.grad_weight) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.cols + kRedX - 1) / kRedX));
    cfg.blockDim = dim3(kRedX * kRedY);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_grad_weight_kernel<T>, (const float *)a.partial, grid, a.cols,
                              static_cast<T *>(a.grad_weight));
}

template <typename T, bool AL> cudaError_t launch_al(const NormArgs &a, cudaStream_t stream) {
    const Config c = config_of(a.cols, Storage<T>::kVec);
    if (c.tpr == 8) return launch_one<T, 8, 1, AL>(a, c.threads, stream);
    if (c.tpr == 32 && c.nv == 1) return launch_one<T, 32, 1, AL>(a, c.threads, stream);
    if (c.tpr == 32 && c.nv == 2) return launch_one<T, 32, 2, AL>(a, c.threads, stream);
    if (c.tpr == 32) return launch_one<T, 32, 4, AL>(a, c.threads, stream);
    return launch_one<T, 0, 16 / Storage<T>::kVec, AL>(a, c.threads, stream);
}

template <typename T> cudaError_t launch_t(const NormArgs &a, cudaStream_t stream) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.h) | reinterpret_cast<uintptr_t>(a.grad_out) |
                           reinterpret_cast<uintptr_t>(a.grad_residual_out) | reinterpret_cast<uintptr_t>(a.weight) |
                           reinterpret_cast<uintptr_t>(a.grad_x) | (uintptr_t)((size_t)a.cols * sizeof(T));
    return bits % 16 == 0 ? launch_al<T, true>(a, stream) : launch_al<T, false>(a, stream);
}

}  // namespace

int norm_backward_partial_rows(int64_t rows, int cols, DType dtype) {
    const Config c = config_of(cols, dtype == DType::F32 ? 4 : 8);
    const int teams = c.tpr ? c.threads / c.tpr : 1;
    const int64_t need = (rows + teams - 1) / teams, most = (int64_t)kSms * c.per_sm;
    return (int)(need < most ? need : most);
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
