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
// Measured (one B200): fp32 12800 x 512 with a gradient of the new residual 20.4
// us (105 MB: 5.1 TB/s; 17.8 us without the weight's gradient, 16.4 us = 6.4 TB/s without a weight), bf16 102400 x 256
// 38.2 us (210 MB: 5.5 TB/s); off 16-byte boundaries fp16 5734 x 4383 73 us (201 MB: 2.8 TB/s; one CTA of 9 warps an
// SM), fp32 4001 x 6001 69 us (384 MB: 5.6 TB/s), by elements fp16 30011 x 521 64 us (125 MB: 2.0 TB/s), 2000 x 601
// 9.5 us; wider than 8192 columns bf16 4096 x 12288 239 us (403 MB: 1.7 TB/s).
#include "dcn_device.h"
#include "dcn_host.h"
#include "dcn_launch.h"
#include "dcn_norm.cuh"

namespace dcnb {
namespace {

constexpr int kTeamThreads = 512;  // CTA of 8-lane and warp teams
constexpr int kSms = 148;

// One row of partial sums of the weight gradient from the CTA's first WARPS warps.  Narrow teams add up pairs of
// warps through shared memory (`sums`, sum_floats()), halving their number each time; 8-lane teams of a warp first
// among themselves.
constexpr int sum_floats(int columns, int warps) { return (warps / 2) * 32 * columns; }  // columns of a thread
template <int TPR, int NV, int VEC, int WARPS, bool ELEMS = false>
__device__ __forceinline__ void store_partial(const NormArgs &a, float2 (&gw)[NV][VEC / 2], float *sums, int t, int tpr,
                                              int shift = 0) {
    float *part = a.partial + (long long)blockIdx.x * a.cols;
    if constexpr (TPR != 0) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        auto sync = [] { asm volatile("bar.sync 1, %0;" ::"r"(WARPS * 32) : "memory"); };
        if (TPR == 8) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j)
#pragma unroll
                    for (int o = 8; o < 32; o <<= 1) {
                        gw[i][j].x += __shfl_xor_sync(0xffffffffu, gw[i][j].x, o);
                        gw[i][j].y += __shfl_xor_sync(0xffffffffu, gw[i][j].y, o);
                    }
        }
        // float2 k of a lane at [k][lane]: neighbouring lanes use neighbouring banks
        float2 *slots = reinterpret_cast<float2 *>(sums);
        constexpr int K = NV * VEC / 2;
        sync();  // whatever was in `sums` has been read
#pragma unroll
        for (int n = WARPS; n > 1;) {
            const int half = (n + 1) / 2;
            if (warp >= half && warp < n) {
#pragma unroll
                for (int k = 0; k < K; ++k) slots[((warp - half) * K + k) * 32 + lane] = gw[k / (VEC / 2)][k % (VEC / 2)];
            }
            sync();
            if (warp < n - half) {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    gw[k / (VEC / 2)][k % (VEC / 2)] =
                        f2_add(gw[k / (VEC / 2)][k % (VEC / 2)], slots[(warp * K + k) * 32 + lane]);
            }
            sync();
            n = half;
        }
        if (warp != 0 || lane >= TPR) return;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int c = ELEMS ? (i * VEC + j) * tpr + t : (t + i * tpr) * VEC + j - shift;
            if (c >= 0 && c < a.cols) part[c] = j % 2 ? gw[i][j / 2].y : gw[i][j / 2].x;
        }
}

template <typename T, int NV, bool SHIFT = false>
__device__ __forceinline__ void load_weight(const NormArgs &a, int t, int tpr, float2 (&w)[NV][Storage<T>::kVec / 2],
                                            float2 (&gw)[NV][Storage<T>::kVec / 2], int shift = 0) {
    constexpr int VEC = Storage<T>::kVec;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const T *weight = static_cast<const T *>(a.weight);
        const int c = (t + i * tpr) * VEC - shift;
        if (a.weight) unpack16x2<T>(SHIFT ? load_any<T>(weight, c, a.cols) : load_cols<T>(weight, c, a.cols), w[i]);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            if (!a.weight) w[i][j] = make_float2(1.0f, 1.0f);
            gw[i][j] = make_float2(0.0f, 0.0f);
        }
    }
}

// The narrowest rows, 16-byte aligned: a vector each for 8 lanes.  The loads of a team's next row are in flight
// while it works on the current one.
template <typename T> __global__ void __launch_bounds__(kTeamThreads, 2) norm_backward_narrow_kernel(const NormArgs a) {
    constexpr int VEC = Storage<T>::kVec, TPR = 8, TEAMS = kTeamThreads / TPR;
    __shared__ __align__(16) float sums[sum_floats(VEC, kTeamThreads / 32)];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = threadIdx.x % TPR, team = threadIdx.x / TPR;
    const T *hp = static_cast<const T *>(a.h), *gyp = static_cast<const T *>(a.grad_out);
    const T *ghp = static_cast<const T *>(a.grad_residual_out);
    float2 w[1][VEC / 2], gw[1][VEC / 2];
    load_weight<T, 1>(a, t, TPR, w, gw);
    const float inv_cols = 1.0f / (float)a.cols;
    const long long step = (long long)gridDim.x * TEAMS;
    uint4 hn, gn, rn;
    float sn = 0.0f;
    auto fetch = [&](long long r) {
        const long long off = r < a.rows ? r * a.cols : 0;
        const int cols = r < a.rows ? a.cols : 0;
        sn = r < a.rows ? a.rstd[r] : 0.0f;
        hn = load_cols<T>(hp + off, t * VEC, cols);
        gn = load_cols<T>(gyp + off, t * VEC, cols);
        if (ghp) rn = load_cols<T>(ghp + off, t * VEC, cols);
    };
    fetch((long long)blockIdx.x * TEAMS + team);
    // every lane of a warp runs the same number of rounds: the shuffles need them all
    for (long long base = (long long)blockIdx.x * TEAMS; base < a.rows; base += step) {
        const long long r = base + team;
        const float rstd = sn;
        float2 xh[VEC / 2], gy[VEC / 2], o[VEC / 2], dot2 = make_float2(0.0f, 0.0f);
        unpack16x2<T>(hn, xh);
        unpack16x2<T>(gn, gy);
        if (ghp) unpack16x2<T>(rn, o);
        fetch(r + step);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            xh[j] = f2_mul(xh[j], make_float2(rstd, rstd));
            const float2 p = f2_mul(gy[j], xh[j]);
            gw[0][j] = f2_add(gw[0][j], p);
            dot2 = f2_fma(p, w[0][j], dot2);
        }
        const float dot = -lanes_reduce<SumOp, TPR>(dot2.x + dot2.y) * inv_cols;
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            const float2 d = f2_fma(xh[j], make_float2(dot, dot), f2_mul(gy[j], w[0][j]));
            o[j] = ghp ? f2_fma(d, make_float2(rstd, rstd), o[j]) : f2_mul(d, make_float2(rstd, rstd));
        }
        if (r < a.rows)
            store_cols<T>(static_cast<T *>(a.grad_x) + r * a.cols, t * VEC, a.cols,
                          pack16<T>(reinterpret_cast<const float *>(o)));
    }
    if (!a.grad_weight) return;
    store_partial<TPR, 1, VEC, kTeamThreads / 32>(a, gw, sums, t, TPR);
}

// Rows at any alignment, by elements: warp or CTA teams of C columns a thread.  Also aligned rows of more than 8192
// columns, which 512 threads of 16 columns do not hold (1024 threads have 64 registers each, of which the staged kernel
// needs up to 128; two slots of three 16-bit rows of 16384 columns would fit the shared memory, of fp32 rows only up to
// some 9600): bf16 4096 x 12288 239 us, 2048 x 16384 149, fp32 230 and 146, 2 to 4 times their floors.  Nothing is loaded ahead: narrow rows take many warps instead, of as few
// columns a lane as hold the row (fp16 100000 x 61 24 us, with 8 columns a lane 59; 300000 x 21 55 against 161).
constexpr int elems_per_sm(int c) { return c <= 4 ? 6 : c <= 8 ? 4 : 2; }
template <typename T, int TPR, int C>
__global__ void __launch_bounds__(TPR == 0 ? 1024 : 256, TPR == 0 ? 1 : elems_per_sm(C))
    norm_backward_elems_kernel(const NormArgs a) {
    constexpr int WARPS = 8;
    __shared__ __align__(16) float sums[TPR == 0 ? 64 : sum_floats(C, WARPS)];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tpr = TPR == 0 ? (int)blockDim.x : TPR;
    const int t = TPR == 0 ? (int)threadIdx.x : (int)threadIdx.x % 32;
    const int teams = TPR == 0 ? 1 : WARPS, team = TPR == 0 ? 0 : (int)threadIdx.x / 32;
    int turn = 0;
    float w[C];
    float2 gw[1][C / 2];
    if (a.weight) load_elems<T, C>(static_cast<const T *>(a.weight), t, tpr, a.cols, w);
#pragma unroll
    for (int k = 0; k < C; ++k) {
        if (!a.weight) w[k] = 1.0f;
        if (k % 2 == 0) gw[0][k / 2] = make_float2(0.0f, 0.0f);
    }
    const float inv_cols = 1.0f / (float)a.cols;
    const long long step = (long long)gridDim.x * teams;
    for (long long r = (long long)blockIdx.x * teams + team; r < a.rows; r += step) {  // the same in the whole team
        const long long off = r * a.cols;
        const float rstd = a.rstd[r];
        float xh[C], gy[C], o[C], dot = 0.0f;
        load_elems<T, C>(static_cast<const T *>(a.h) + off, t, tpr, a.cols, xh);
        load_elems<T, C>(static_cast<const T *>(a.grad_out) + off, t, tpr, a.cols, gy);
        if (a.grad_residual_out) load_elems<T, C>(static_cast<const T *>(a.grad_residual_out) + off, t, tpr, a.cols, o);
#pragma unroll
        for (int k = 0; k < C; ++k) {
            xh[k] *= rstd;
            const float p = gy[k] * xh[k];
            if (k % 2) gw[0][k / 2].y += p;
            else gw[0][k / 2].x += p;
            dot = fmaf(p, w[k], dot);
        }
        dot = -team_reduce<SumOp, TPR>(dot, sums, turn) * inv_cols;
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const float d = fmaf(xh[k], dot, gy[k] * w[k]);
            const float gx = a.grad_residual_out ? fmaf(d, rstd, o[k]) : d * rstd;
            if (k * tpr + t < a.cols) static_cast<T *>(a.grad_x)[off + k * tpr + t] = from_f32<T>(gx);
        }
    }
    if (!a.grad_weight) return;
    store_partial<TPR, 1, C, WARPS, true>(a, gw, sums, t, tpr);
}

// A row's products from its staged tensors: xh and grad_out in registers, the weight gradient, and this thread's part
// of sum(g * xh).
template <typename T, int NV, bool SHIFT>
__device__ __forceinline__ float staged_row(const RowVecs<T, SHIFT, true> &in, const NormArgs &a, const unsigned char *h,
                                            const unsigned char *g, int t, int tpr,
                                            float rstd, const float2 (&w)[NV][Storage<T>::kVec / 2],
                                            float2 (&xh)[NV][Storage<T>::kVec / 2], float2 (&gy)[NV][Storage<T>::kVec / 2],
                                            float2 (&gw)[NV][Storage<T>::kVec / 2]) {
    constexpr int VEC = Storage<T>::kVec;
    float2 dot = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * tpr) * VEC - in.shift;
        unpack16x2<T>(in.load(h, a.h, i, c), xh[i]);
        unpack16x2<T>(in.load(g, a.grad_out, i, c), gy[i]);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            xh[i][j] = f2_mul(xh[i][j], make_float2(rstd, rstd));
            const float2 p = f2_mul(gy[i][j], xh[i][j]);
            gw[i][j] = f2_add(gw[i][j], p);
            dot = f2_fma(p, w[i][j], dot);
        }
    }
    return dot.x + dot.y;
}

// grad_x of the row; `r` the staged gradient of the new residual, or nullptr.
template <typename T, int NV, bool SHIFT>
__device__ __forceinline__ void staged_output(const RowVecs<T, SHIFT, true> &in, const NormArgs &a, const unsigned char *r, int t,
                                              int tpr, float rstd, float mean, const float2 (&w)[NV][Storage<T>::kVec / 2],
                                              const float2 (&xh)[NV][Storage<T>::kVec / 2],
                                              const float2 (&gy)[NV][Storage<T>::kVec / 2]) {
    constexpr int VEC = Storage<T>::kVec;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * tpr) * VEC - in.shift;
        float2 o[VEC / 2];
        if (r) unpack16x2<T>(in.load(r, a.grad_residual_out, i, c), o);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            const float2 d = f2_fma(xh[i][j], make_float2(-mean, -mean), f2_mul(gy[i][j], w[i][j]));
            o[j] = r ? f2_fma(d, make_float2(rstd, rstd), o[j]) : f2_mul(d, make_float2(rstd, rstd));
        }
        store_vec<T, SHIFT>(static_cast<T *>(a.grad_x) + in.off, c, in.cols, pack16<T>(reinterpret_cast<const float *>(o)));
    }
}

constexpr int kMaxSlots = 8;

// Rows of up to 512 columns, 16-byte aligned: WARPS rows at a time, one per warp, are contiguous in memory, and a
// further warp copies such tiles of the two or three tensors into a ring in shared memory, one bulk copy each
// (copies of single rows measured 51 us on bf16 102400 x 256, tiles 38.2 us).
template <typename T, int NV, int WARPS, int CTAS>
__global__ void __launch_bounds__((WARPS + 1) * 32, CTAS)
    norm_backward_tiles_kernel(const NormArgs a, int slots, unsigned int *err) {
    constexpr int VEC = Storage<T>::kVec;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ __align__(8) uint64_t bars[2 * kMaxSlots];  // full, empty
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, t = threadIdx.x & 31;
    const uint32_t row_bytes = (uint32_t)a.cols * sizeof(T), tile_bytes = WARPS * row_bytes;
    const uint32_t slot_bytes = (a.grad_residual_out ? 3 : 2) * tile_bytes;
    const uint32_t full = smem_u32(bars), empty = full + 8 * kMaxSlots;
    if (threadIdx.x == 0) {
        for (int i = 0; i < slots; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, WARPS);
        }
        fence_mbar_init();
    }
    __syncthreads();
    const long long tiles = (a.rows + WARPS - 1) / WARPS;
    int s = 0;
    uint32_t phase = 0;
    if (warp == WARPS) {
        if (t == 0) {
            for (long long i = blockIdx.x; i < tiles; i += gridDim.x) {
                // (the first pass over the ring waits for the phase before the first, which counts as complete)
                if (!mbar_wait_bounded(empty + 8 * s, phase ^ 1u, kRowWaitNs)) {
                    atomicOr(err, kDevErrTmaTimeout);
                    break;
                }
                const long long r = i * WARPS, off = r * a.cols, left = a.rows - r;
                const uint32_t bytes = (uint32_t)(left < WARPS ? left : WARPS) * row_bytes;
                const uint32_t bar = full + 8 * s, dst = smem_u32(ring) + s * slot_bytes;
                mbar_arrive_expect_tx(bar, (a.grad_residual_out ? 3 : 2) * bytes);
                bulk_load(dst, static_cast<const T *>(a.h) + off, bytes, bar);
                bulk_load(dst + tile_bytes, static_cast<const T *>(a.grad_out) + off, bytes, bar);
                if (a.grad_residual_out)
                    bulk_load(dst + 2 * tile_bytes, static_cast<const T *>(a.grad_residual_out) + off, bytes, bar);
                if (++s == slots) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        return;
    }
    float2 w[NV][VEC / 2], gw[NV][VEC / 2];
    load_weight<T, NV>(a, t, 32, w, gw);
    const float inv_cols = 1.0f / (float)a.cols;
    const long long step = (long long)gridDim.x * WARPS;
    long long r = (long long)blockIdx.x * WARPS + warp;
    float next_rstd = r < a.rows ? __ldg(a.rstd + r) : 0.0f;
    for (long long i = blockIdx.x; i < tiles; i += gridDim.x, r += step) {
        const float rstd = next_rstd;
        next_rstd = r + step < a.rows ? __ldg(a.rstd + r + step) : 0.0f;
        if (!mbar_wait_bounded(full + 8 * s, phase, kRowWaitNs)) {
            if (t == 0) give_up(full, s, phase, slots, err);
            __syncwarp();
            break;
        }
        if (r < a.rows) {
            const unsigned char *base = ring + s * slot_bytes + warp * row_bytes;
            float2 xh[NV][VEC / 2], gy[NV][VEC / 2];
            const RowVecs<T, false, true> in{a.cols, r * a.cols};
            float dot = staged_row<T, NV, false>(in, a, base, base + tile_bytes, t, 32, rstd, w, xh, gy, gw);
            dot = lanes_reduce<SumOp, 32>(dot) * inv_cols;
            staged_output<T, NV, false>(in, a, a.grad_residual_out ? base + 2 * tile_bytes : nullptr, t, 32, rstd, dot, w, xh,
                                        gy);
        }
        __syncwarp();
        if (t == 0) mbar_arrive(empty + 8 * s);
        if (++s == slots) {
            s = 0;
            phase ^= 1;
        }
    }
    if (!a.grad_weight) return;
    // every tile has been read: the ring is free (two slots of WARPS rows hold more than the sums of WARPS / 2)
    store_partial<32, NV, VEC, WARPS>(a, gw, reinterpret_cast<float *>(ring), t, 32);
}

// Wider rows of up to 8192 columns: a CTA of 16 columns a thread per row, each row of the tensors copied into the ring
// by one bulk copy (rows off 16-byte boundaries by vectors of the aligned grid, dcn_norm.cuh).  The slot of a row is
// handed back behind the barrier of the next row's reduction, when the whole CTA is past its output.
template <typename T, bool SHIFT>
__global__ void __launch_bounds__(512, 1) norm_backward_wide_kernel(const NormArgs a, int slots, unsigned int *err) {
    constexpr int VEC = Storage<T>::kVec, NV = 16 / VEC;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ float red[64];
    __shared__ __align__(8) uint64_t bars_s[kMaxSlots];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = threadIdx.x, tpr = blockDim.x;
    const long long total = a.rows * a.cols;
    // SHIFT: the grid is a multiple of VEC, or no CTA has two rows
    const int sh = SHIFT ? shift_of_rows<T>(a.h, blockIdx.x, a.cols) : 0, nvec = (a.cols + sh + VEC - 1) / VEC;
    const uint32_t row_bytes = (uint32_t)nvec * 16, slot_bytes = (a.grad_residual_out ? 3 : 2) * row_bytes;
    const uint32_t bars = smem_u32(bars_s);
    int turn = 0;
    if (t == 0) {
        for (int i = 0; i < slots; ++i) mbar_init(bars + 8 * i, 1);
        fence_mbar_init();
    }
    __syncthreads();
    auto stage = [&](long long r, int s) {  // by thread 0
        if (r >= a.rows) return;
        // without a vector that reaches out of the tensor at either end
        const long long first_vec = r * a.cols - sh;
        const int skip = SHIFT && first_vec < 0, n = nvec - skip - (SHIFT && first_vec + (long long)nvec * VEC > total);
        const long long e = first_vec + skip * VEC;
        const uint32_t bar = bars + 8 * s, dst = smem_u32(ring) + s * slot_bytes + 16 * skip;
        mbar_arrive_expect_tx(bar, (a.grad_residual_out ? 48u : 32u) * n);
        bulk_load(dst, static_cast<const T *>(a.h) + e, 16u * n, bar);
        bulk_load(dst + row_bytes, static_cast<const T *>(a.grad_out) + e, 16u * n, bar);
        if (a.grad_residual_out)
            bulk_load(dst + 2 * row_bytes, static_cast<const T *>(a.grad_residual_out) + e, 16u * n, bar);
    };
    const long long step = gridDim.x, first = blockIdx.x;
    if (t == 0)
        for (int i = 0; i < slots; ++i) stage(first + i * step, i);
    float2 w[NV][VEC / 2], gw[NV][VEC / 2];
    load_weight<T, NV, SHIFT>(a, t, tpr, w, gw, sh);
    RowVecs<T, SHIFT, true> in{a.cols, 0};
    in.init(sh, nvec, t, tpr);
    const float inv_cols = 1.0f / (float)a.cols;
    float next_rstd = first < a.rows ? __ldg(a.rstd + first) : 0.0f;
    int s = 0;
    uint32_t phase = 0;
    for (long long r = first; r < a.rows; r += step) {
        const float rstd = next_rstd;
        next_rstd = r + step < a.rows ? __ldg(a.rstd + r + step) : 0.0f;
        if (!mbar_wait_bounded(bars + 8 * s, phase, kRowWaitNs)) {
            give_up(bars, s, phase, slots, err);
            return;
        }
        const unsigned char *base = ring + s * slot_bytes;
        float2 xh[NV][VEC / 2], gy[NV][VEC / 2];
        in.at(r, total);
        float dot = staged_row<T, NV, SHIFT>(in, a, base, base + row_bytes, t, tpr, rstd, w, xh, gy, gw);
        dot = team_reduce<SumOp, 0>(dot, red, turn) * inv_cols;
        if (t == 0 && r != first) stage(r + (slots - 1) * step, s ? s - 1 : slots - 1);
        staged_output<T, NV, SHIFT>(in, a, a.grad_residual_out ? base + 2 * row_bytes : nullptr, t, tpr, rstd, dot, w, xh,
                                    gy);
        if (++s == slots) {
            s = 0;
            phase ^= 1;
        }
    }
    if (!a.grad_weight) return;
    store_partial<0, NV, VEC, 0>(a, gw, red, t, tpr, sh);
}

// grad_weight[c] = sum over the CTAs of the first kernel, in a fixed order: 8
// columns (one 32-byte sector of a row of partial sums) and Y threads along the
// rows, so that a thread has a few loads and all of them in flight at once.
constexpr int kRedX = 8;
template <typename T, int Y>
__global__ void __launch_bounds__(kRedX *Y) norm_grad_weight_kernel(const float *partial, int n, int cols, T *out) {
    __shared__ float s[Y / 4][kRedX];
    const int x = threadIdx.x % kRedX, y = threadIdx.x / kRedX, c = blockIdx.x * kRedX + x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float v = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int k = y; k < n; k += Y) v += __ldcg(partial + (long long)k * cols + c);
    }
    // the 4 threads of a warp that share a column, then the warps
    v += __shfl_xor_sync(0xffffffffu, v, 8);
    v += __shfl_xor_sync(0xffffffffu, v, 16);
    s[y / 4][x] = v;
    __syncthreads();
    if (y == 0 && c < cols) {
#pragma unroll
        for (int k = 1; k < Y / 4; ++k) v += s[k][x];
        out[c] = from_f32<T>(v);
    }
}

// How rows are worked on: `threads` of a CTA, `rows` at a time, `per_sm` CTAs on an SM.
enum Route { kNarrow, kTiles, kWide, kElems };
struct Config {
    Route route;
    int nv, threads, rows, per_sm;  // nv vectors (kElems: columns) a thread
    int shift;                      // 0, or the largest shift of a row, VEC - 1
};
// How all tensors' rows lie: on 16-byte boundaries, off them by the same in all tensors, or in any way.
enum Lie { kAligned, kInStep, kAnyhow };
Config config_of(int cols, int vec, Lie lie) {
    const bool aligned = lie == kAligned;
    const int nvec = (cols + vec - 1) / vec, nv16 = 16 / vec;
    if (aligned && nvec <= 8) return {kNarrow, 1, kTeamThreads, kTeamThreads / 8, 2, 0};
    if (aligned && cols <= 512) {
        // columns a thread -> registers -> warps: 72 registers for two CTAs of 13 warps, 112 for one of 17
        const int nv = nvec <= 32 ? 1 : nvec <= 64 ? 2 : 4;
        if (nv * vec <= 8) return {kTiles, nv, 13 * 32, 12, 2, 0};
        return {kTiles, nv, 17 * 32, 16, 1, 0};
    }
    const int shift = aligned ? 0 : vec - 1, span = cols + shift;  // columns of a row's vectors
    // fp32 rows in step gain from 2048 columns on (9093 x 2047 54.7 us against 51.8 by elements, 7001 x 3001 59.5 against
    // 64.4, 4001 x 6001 68 against 90), 16 bits from 1024 (fp16 20011 x 1101 63 against 67, 4001 x 6001 57 against 95;
    // below, 30011 x 769 57 against 74, but 2000 x 1001 15 against 11)
    if (span <= 8192 && (aligned || (lie == kInStep && cols > (vec == 4 ? 2048 : 1024)))) {
        const int wide = ((span + 15) / 16 + 31) / 32 * 32;  // threads of a CTA for a row, 16 columns each
        // 16 bits up to 1024 columns: 30011 x 600 53 us in tiles (32 columns a lane), 34 so; fp32 is at the copy rate with 4
        const int cap = vec == 8 && cols <= 1024 ? 8 : 4;
        int per_sm = 512 / wide < cap ? 512 / wide : cap;
        // fewer CTAs where two staged rows of three tensors would not fit their share of the shared memory
        while (per_sm > 1 && 2 * 3 * (span + vec - 1) / vec * 16 > staged_budget(per_sm)) --per_sm;
        return {kWide, nv16, wide, 1, per_sm, shift};
    }
    for (int c = 2; c <= 16; c *= 2)
        if (cols <= 32 * c) return {kElems, c, 256, 8, elems_per_sm(c), 0};
    const int c = cols <= 8192 ? 8 : 16, threads = ((cols + c - 1) / c + 31) / 32 * 32;  // at most 1024
    return {kElems, c, threads, 1, 1024 / threads < 8 ? 1024 / threads : 8, 0};
}

int grid_of(int64_t rows, const Config &c) {
    const int64_t need = (rows + c.rows - 1) / c.rows;
    int64_t most = (int64_t)kSms * c.per_sm;
    // narrow rows' many CTAs: four rows each at least, or their partial sums cost more than they give (fp16 1000 x 600 9.2 us
    // with a row each, 6.9 so)
    if (c.route == kWide && c.per_sm > 4 && most > rows / 4) most = rows / 4 > kSms ? rows / 4 : kSms;
    most -= most % (c.shift + 1);  // shifted: a CTA's rows have the same shift
    return (int)(need < most ? need : most);
}

template <typename T> cudaError_t launch_grad_weight(const NormArgs &a, int n, cudaStream_t stream) {
    if (!a.grad_weight) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.cols + kRedX - 1) / kRedX));
    const bool many = n > 32;  // rows of partial sums
    cfg.blockDim = dim3(kRedX * (many ? 64 : 8));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, many ? norm_grad_weight_kernel<T, 64> : norm_grad_weight_kernel<T, 8>,
                              (const float *)a.partial, n, a.cols, static_cast<T *>(a.grad_weight));
}

template <typename K> cudaError_t launch_plain(K kern, const NormArgs &a, const Config &c, cudaStream_t stream) {
    kern<<<grid_of(a.rows, c), c.threads, 0, stream>>>(a);
    return cudaGetLastError();
}

// Staged launch: as many slots as fit, at least two.
template <typename K>
cudaError_t launch_staged(K kern, const NormArgs &a, const Config &c, int budget, int es, std::atomic<bool> (&ok)[kMaxDev],
                          const DeviceInfo *dev, cudaStream_t stream) {
    const int row_bytes = ((a.cols + c.shift) * es + 15) / 16 * 16;  // the tiles' rows are multiples of 16 bytes
    const int slot = row_bytes * (a.grad_residual_out ? 3 : 2) * c.rows;
    int slots = budget / slot;
    if (slots > kMaxSlots) slots = kMaxSlots;
    const cudaError_t e = allow_smem(kern, staged_budget(1), ok);
    if (e != cudaSuccess) return e;
    kern<<<grid_of(a.rows, c), c.threads, slots * slot, stream>>>(a, slots, dev->err);
    return cudaGetLastError();
}

template <typename T, int NV, int WARPS, int CTAS>
cudaError_t launch_tiles(const NormArgs &a, const Config &c, const DeviceInfo *dev, cudaStream_t stream) {
    static std::atomic<bool> ok[kMaxDev];
    return launch_staged(norm_backward_tiles_kernel<T, NV, WARPS, CTAS>, a, c, staged_budget(CTAS),
                         (int)sizeof(T), ok, dev, stream);
}

template <typename T> cudaError_t launch_rows(const NormArgs &a, const Config &c, cudaStream_t stream) {
    constexpr int VEC = Storage<T>::kVec;
    const DeviceInfo *dev = device_info();
    if (!dev) return cudaErrorNotSupported;
    switch (c.route) {
        case kNarrow: return launch_plain(norm_backward_narrow_kernel<T>, a, c, stream);
        case kTiles:
            if (c.nv == 1) return launch_tiles<T, 1, 12, 2>(a, c, dev, stream);
            if constexpr (VEC == 4) {
                if (c.nv == 2) return launch_tiles<T, 2, 12, 2>(a, c, dev, stream);
                return launch_tiles<T, 4, 16, 1>(a, c, dev, stream);
            } else {
                return launch_tiles<T, 2, 16, 1>(a, c, dev, stream);
            }
        case kWide: {
            static std::atomic<bool> ok[kMaxDev], shift_ok[kMaxDev];
            return c.shift ? launch_staged(norm_backward_wide_kernel<T, true>, a, c, staged_budget(c.per_sm), (int)sizeof(T),
                                           shift_ok, dev, stream)
                           : launch_staged(norm_backward_wide_kernel<T, false>, a, c, staged_budget(c.per_sm), (int)sizeof(T),
                                           ok, dev, stream);
        }
        case kElems:
            if (c.rows > 1)
                return c.nv == 2   ? launch_plain(norm_backward_elems_kernel<T, 32, 2>, a, c, stream)
                       : c.nv == 4 ? launch_plain(norm_backward_elems_kernel<T, 32, 4>, a, c, stream)
                       : c.nv == 8 ? launch_plain(norm_backward_elems_kernel<T, 32, 8>, a, c, stream)
                                   : launch_plain(norm_backward_elems_kernel<T, 32, 16>, a, c, stream);
            return c.nv == 16 ? launch_plain(norm_backward_elems_kernel<T, 0, 16>, a, c, stream)
                              : launch_plain(norm_backward_elems_kernel<T, 0, 8>, a, c, stream);
    }
    return cudaErrorInvalidValue;
}

template <typename T> cudaError_t launch_t(const NormArgs &a, cudaStream_t stream) {
    const uintptr_t h = reinterpret_cast<uintptr_t>(a.h), gy = reinterpret_cast<uintptr_t>(a.grad_out);
    const uintptr_t gh = reinterpret_cast<uintptr_t>(a.grad_residual_out), gx = reinterpret_cast<uintptr_t>(a.grad_x);
    const uintptr_t bits = h | gy | gh | gx | reinterpret_cast<uintptr_t>(a.weight) | (uintptr_t)((size_t)a.cols * sizeof(T));
    const bool in_step = (h ^ gy) % 16 == 0 && (h ^ gx) % 16 == 0 && (!gh || (h ^ gh) % 16 == 0);
    const Config c = config_of(a.cols, Storage<T>::kVec, bits % 16 == 0 ? kAligned : in_step ? kInStep : kAnyhow);
    const cudaError_t e = launch_rows<T>(a, c, stream);
    return e != cudaSuccess ? e : launch_grad_weight<T>(a, grid_of(a.rows, c), stream);
}

}  // namespace

int norm_backward_partial_rows(int64_t rows, int cols, DType dtype) {
    // how the tensors lie is not known yet
    const int vec = dtype == DType::F32 ? 4 : 8;
    int most = 0;
    for (const Lie lie : {kAligned, kInStep, kAnyhow}) {
        const int n = grid_of(rows, config_of(cols, vec, lie));
        if (n > most) most = n;
    }
    return most;
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
