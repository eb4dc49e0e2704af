// Internal launcher interface between the C-ABI layer (dcn_abi.cu) and the
// kernels.  Arguments are validated by the ABI layer before any launcher runs.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dcnb {

enum class DType : int { F32 = 0, F16 = 1, BF16 = 2 };

// Largest K for which the softmax-mode backward keeps per-point gradients.
constexpr int kMaxSoftmaxK = 49;

struct CoreArgs {
    const void *x;
    const void *offset;
    const void *mask;
    void *out;              // forward output
    const void *grad_out;   // backward only
    void *grad_x;           // backward only
    void *grad_offset;      // backward only
    void *grad_mask;        // backward only
    int B, H, W, G, C, kh, kw, sh, sw, ph, pw, dh, dw, Ho, Wo;
    float offset_scale;
    bool softmax;
    DType dtype;
};

// Forward core followed by its pointwise projection (fp16/bf16 only).
struct ProjArgs {
    CoreArgs core;       // core.out is the projected output [B, Ho, Wo, Cout]
    const void *weight;  // [Cout, G*C], or [Cout, K, G*C] when per_point
    const void *bias;    // [Cout] or nullptr
    int Cout;
    bool per_point;      // deformable convolution: a dense weight per kernel point
};

struct AggArgs {
    const void *feat;
    const int32_t *spatial_shape;
    const int32_t *scale_start;
    const float *loc;
    const void *weights;
    void *out;
    const void *grad_out;   // backward only
    void *grad_feat;        // backward only
    float *grad_loc;        // backward only
    void *grad_weights;     // backward only
    int B, cams, scales, rows, A, P, G, C;
    DType dtype;
};

struct RoiArgs {
    const void *x;       // [B, H, W, C]
    const float *rois;   // [N, 5]
    const float *offset; // [N, PH, PW, 2]
    void *out;           // [N, PH, PW, C]
    int B, H, W, C, N, PH, PW, S;
    float spatial_scale, gamma;
    DType dtype;
};

// 8-bit output kinds of the norm (dcn_quant8 of the ABI).
enum : int { kQuantNone = 0, kQuantE4M3 = 1, kQuantInt8 = 2 };

// Residual addition + root-mean-square norm over rows of `cols` values.
struct NormArgs {
    const void *x, *residual, *weight;  // forward; residual and weight may be nullptr
    void *residual_out, *out, *out8;    // forward; out or out8 may be nullptr
    float *scale;                       // forward: [rows] or [rows, groups]
    float *rstd;                        // [rows]: written by the forward (or nullptr), read by the backward
    const void *h, *grad_out, *grad_residual_out;  // backward; grad_residual_out may be nullptr
    void *grad_x, *grad_weight;         // backward; grad_weight may be nullptr
    float *partial;                     // backward: [norm_backward_partial_rows(), cols] partial weight gradients
    int64_t rows;
    int cols;
    float eps;
    int quant, group, groups;           // group: 0 or 128 columns per scale
    DType dtype;
};

// Global gradient norm and clipping over tables of tensors (host arrays).
struct ClipArgs {
    const void *const *grads;
    void *const *outs;         // nullptr: in place
    const int64_t *numel;
    const int32_t *dtypes, *out_dtypes;
    int num_tensors;
    bool inf, clip;            // maximum norm instead of the 2-norm; clip after the norm
    float max_norm, eps;
    float *norm;
    double *partial;           // grad_clip_partials(num_tensors) values
};

// Pointwise projection with low-rank adapters of many requests (fp16/bf16).
struct AdapterArgs {
    const void *x, *weight, *bias;  // [rows, cin], [cout, cin], [cout] or nullptr
    const void *a, *b;              // [adapters, rank, cin], [adapters, cout, rank]
    const float *scale;             // [adapters] or nullptr (ones)
    const int32_t *start, *which;   // [requests + 1] row starts, [requests] adapters
    void *out;                      // [rows, cout]
    void *workspace;
    size_t workspace_bytes;         // proj_adapters_workspace() at least, proj_adapters_workspace_full() for one pass
    int64_t rows;
    int cin, cout, rank, adapters, requests;
    DType dtype;
};

// Each launcher enqueues its kernel(s) on `stream` and returns the
// cudaGetLastError() of the launch.
cudaError_t launch_core_forward_generic(const CoreArgs &a, cudaStream_t stream);
cudaError_t launch_core_backward_generic(const CoreArgs &a, cudaStream_t stream);
// Staged backward (TMA row bands, per-tap records) for fp32 storage with 128-byte
// groups and K <= 9; *handled stays false for other shapes.
cudaError_t launch_core_backward_staged(const CoreArgs &a, cudaStream_t stream, bool *handled);
// Shared-memory path; sets *handled = false (and launches nothing) when the
// problem does not fit it.
cudaError_t launch_core_forward_plane(const CoreArgs &a, cudaStream_t stream, bool *handled);
// Reads and clears the device error word that bounded waits set (bit 0:
// a TMA wait ran out).  Synchronous.
cudaError_t take_device_error(unsigned int *value);
// One thread waits (bounded by limit_ns) on an mbarrier nothing arrives on.
cudaError_t launch_bounded_wait_selftest(long long limit_ns, cudaStream_t stream);
// Fused core + projection (tcgen05 GEMM on the core tile in shared memory).
cudaError_t launch_core_forward_proj(const ProjArgs &a, cudaStream_t stream);
// out[p, o] = bias[o] + sum_j core[p, j] * weight[o, j] on the tensor cores (fp16/bf16;
// core [P, KD], weight [Cout, KD], out [P, Cout]; KD a multiple of 64, Cout of 8 up to 512).
cudaError_t launch_proj_gemm(const void *core, const void *weight, const void *bias, void *out, long long P, int KD,
                             int Cout, DType dtype, cudaStream_t stream);
cudaError_t launch_agg_forward(const AggArgs &a, cudaStream_t stream);
// Anchor-wide aggregation kernels (all groups per CTA); sets *handled = false
// (and launches nothing) when the feature row width does not fit them.
cudaError_t launch_agg_wide(const AggArgs &a, bool bwd, cudaStream_t stream, bool *handled);
cudaError_t launch_agg_backward(const AggArgs &a, cudaStream_t stream);
cudaError_t launch_roi_pool_forward(const RoiArgs &a, cudaStream_t stream);
cudaError_t launch_norm_forward(const NormArgs &a, cudaStream_t stream);
// The backward, and the rows of partial weight gradients that it needs.
cudaError_t launch_norm_backward(const NormArgs &a, cudaStream_t stream);
int norm_backward_partial_rows(int64_t rows, int cols, DType dtype);
// The norm, with clipping where a.clip, and the partial results that it needs.
cudaError_t launch_grad_clip(const ClipArgs &a, cudaStream_t stream);
int64_t grad_clip_partials(int num_tensors);
cudaError_t launch_proj_adapters(const AdapterArgs &a, cudaStream_t stream);
size_t proj_adapters_workspace(const AdapterArgs &a);
size_t proj_adapters_workspace_full(const AdapterArgs &a);

}  // namespace dcnb
