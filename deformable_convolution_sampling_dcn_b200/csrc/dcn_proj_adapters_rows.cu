// Projection with low-rank adapters, few rows (at most 256): single tokens of
// many requests, short prompts.
//   t[m, :] = scale[a] * A[a] x[m]             a = adapter of row m's request
//   y[m, n] = bias[n] + sum_k W[n, k] x[m, k] + sum_j B[a][n, j] t[m, j]
//
// Bound: the weight, which is read once whatever the rows are.
//
// STREAM: the weight's 128 x 64 blocks are dealt out to one CTA per SM in
// contiguous runs, so every SM streams the same number of bytes whatever the
// sizes are; a run may end inside a tile of 128 channels and the next one go
// on there.  Warp 0 loads the blocks and the matching blocks of x by TMA
// (128-byte swizzle, zero fill past every edge) through a ring of up to eight
// stages, about the whole run of an SM, and one thread of warp 1 multiplies
// them by tcgen05.mma with the weight as the 128-row operand and the rows of x
// as the narrow one.  Warps 2..9 meanwhile form t in fp32, one (row, rank) pair
// per warp at a time, straight from device memory; then warps 2..5 store each
// finished or unfinished tile as fp32 partial sums.
//
// COMBINE, a programmatic dependent, has one warp for 16 to 128 channels of a
// row, as many as 8 loads of the warp cover of B.  It loads its rows of B before
// it waits for STREAM, then adds the partial sums in a fixed order, the adapter
// term and the bias, and rounds once.
//
// Measured (one B200): bf16 48 rows 4096 -> 4096, rank 16, 32 adapters 14.6 us
// (43 MB: 2.9 TB/s), fp16 8 rows 512 -> 512 6.2 us.  mma.sync over a cluster that
// meets in distributed shared memory took 30 us on the first, the adapters' A as
// further tiles of the stream 27 us (its boxes are 2 KB).
#include <cudaTypedefs.h>

#include <type_traits>

#include "dcn_device.h"
#include "dcn_proj_adapters.cuh"
#include "dcn_tcgen05.cuh"

namespace dcnb {
namespace {

constexpr int kTN = 128;  // channels of a tile
constexpr int kBK = 64;
constexpr int kWBytes = kTN * kBK * 2;
constexpr int kTWarps = 8;  // warps 2..9 form t, 2..5 of them store
constexpr int kThreads = (2 + kTWarps) * 32;
constexpr int kMaxStages = 8;
constexpr int kSms = 148;

struct SmallParams {
    AdapterArgs a;
    float *t;          // [rows, rank]
    float *partial;    // [ctas + tiles][mpad][128]: CTA c's part of tile i at c + i
    unsigned int *err;
    int mpad;          // rows rounded up to 16
    int kb, tiles;     // blocks of the contraction, tiles of channels
    int ctas;          // runs of blocks
    int stages, tmem_cols;
};

// Adapter of row m (-1: none; -2: the row belongs to no request), by a whole warp.
__device__ __forceinline__ int adapter_of_row(const AdapterArgs &a, int m, int *raw) {
    const int lane = threadIdx.x & 31;
    constexpr int kNear = 256;  // as many as rows: where there are more, some are empty
    for (int s0 = 0; s0 < min(a.requests, kNear); s0 += 128) {
        int lo[4], hi[4], ad[4];  // 128 requests in flight: one round trip for most tables
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = s0 + 32 * i + lane;
            const bool in = s < a.requests;
            lo[i] = in ? a.start[s] : 0;
            hi[i] = in ? a.start[s + 1] : 0;
            ad[i] = in ? a.which[s] : -1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned hit = __ballot_sync(0xffffffffu, lo[i] <= m && m < hi[i]);
            if (hit) {
                const int v = __shfl_sync(0xffffffffu, ad[i], __ffs((int)hit) - 1);
                *raw = v;
                return v >= 0 && v < a.adapters ? v : -1;
            }
        }
    }
    *raw = -1;
    if (a.requests <= kNear) return -2;
    // the first of the others that ends behind row m (a table filled up with empty requests may be long)
    const int s = kNear + warp_first(a.requests - kNear, [&](int i) { return a.start[kNear + i + 1] > m; });
    if (s == a.requests || a.start[s] > m) return -2;
    *raw = a.which[s];
    return adapter_of(a.which, s, a.adapters);
}

// The blocks of CTA c of n: [total * c / n, total * (c + 1) / n).  At most 1024 x 512 blocks and 148 CTAs: the
// products stay far below 2^31.
__device__ __forceinline__ int run_begin(int total, int c, int n) { return total * c / n; }
// The CTA that has block u.
__device__ __forceinline__ int run_of(int total, int u, int n) { return ((u + 1) * n - 1) / total; }

// t[m, r .. r + RK) by one warp.
template <typename T, int RK>
__device__ __forceinline__ void shrink_rows(const AdapterArgs &a, float *tout, int m, int r, int ad) {
    const int lane = threadIdx.x & 31;
    const T *x = static_cast<const T *>(a.x) + (long long)m * a.cin;
    const T *w = static_cast<const T *>(a.a) + ((long long)ad * a.rank + r) * a.cin;
    float acc[RK];
#pragma unroll
    for (int i = 0; i < RK; ++i) acc[i] = 0.0f;
    constexpr int D = RK == 1 ? 8 : 2;  // steps whose loads are in flight together
    for (int k0 = lane * 8; k0 < a.cin + lane * 8; k0 += 256 * D) {
        uint4 xv[D], wv[D][RK];
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int k = k0 + 256 * d;
            const bool in = k < a.cin;
            xv[d] = in ? ld_nc16(x + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < RK; ++i)
                wv[d][i] = in ? ld_nc16(w + (long long)i * a.cin + k) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int d = 0; d < D; ++d) {
            float f[8];
            unpack16<T>(xv[d], f);
#pragma unroll
            for (int i = 0; i < RK; ++i) {
                float g[8];
                unpack16<T>(wv[d][i], g);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[i] = fmaf(f[j], g[j], acc[i]);
            }
        }
    }
    const float mul = a.scale ? a.scale[ad] : 1.0f;
#pragma unroll
    for (int i = 0; i < RK; ++i) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
        if (lane == 0) tout[(long long)m * a.rank + r + i] = acc[i] * mul;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    adapters_rows_stream(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                         const SmallParams p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int sbytes = kWBytes + p.mpad * kBK * 2;  // mpad a multiple of 16: a multiple of 1 KB
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + p.stages * sbytes);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * kMaxStages + 5);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kMaxStages, accf0 = empty0 + 8 * kMaxStages;
    const uint32_t acce0 = accf0 + 16, drain = acce0 + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int total = p.kb * p.tiles;
    // CTAs past the runs only help with t
    const int u0 = (int)blockIdx.x < p.ctas ? run_begin(total, blockIdx.x, p.ctas) : 0;
    const int u1 = (int)blockIdx.x < p.ctas ? run_begin(total, blockIdx.x + 1, p.ctas) : 0;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(accf0 + 8 * i, 1);
            mbar_init(acce0 + 8 * i, 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(p.tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ---- producer
        if (lane == 0) {
            uint32_t s = 0, pass = 0;
            int issued = 0, tile = u0 / p.kb, kb = u0 % p.kb;
            bool ok = true;
            for (int u = u0; u < u1 && ok; ++u) {
                if (pass >= 1 && !wait_or_abort(empty0 + 8 * s, (pass - 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(full0 + 8 * s, (uint32_t)sbytes);
                unsigned char *st = ring + s * sbytes;
                tma_load_2d(smem_u32(st), &wmap, full0 + 8 * s, kb * kBK, tile * kTN);
                tma_load_2d(smem_u32(st + kWBytes), &xmap, full0 + 8 * s, kb * kBK, 0);
                ++issued;
                if (++s == (uint32_t)p.stages) {
                    s = 0;
                    ++pass;
                }
                if (++kb == p.kb) {
                    kb = 0;
                    ++tile;
                }
            }
            if (!ok) raise_abort(abort_flag, p.err);
            // the last load of every stage has landed before the CTA may exit
            for (int j = issued - 1; j >= 0 && j >= issued - p.stages; --j)
                mbar_wait_bounded(full0 + 8 * (uint32_t)(j % p.stages), (uint32_t)(j / p.stages) & 1, kTcWaitNs);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- one thread issues the products
        if (lane == 0) {
            const uint32_t idesc = instr_desc_f16(std::is_same<T, __nv_bfloat16>::value ? 1 : 0, p.mpad);
            const uint64_t a0 = smem_desc_sw128(smem_u32(ring)), b0 = smem_desc_sw128(smem_u32(ring + kWBytes));
            const uint32_t sstep = (uint32_t)sbytes >> 4;
            uint32_t s = 0, ph = 0;
            int local = 0;
            bool ok = true, issued = false;
            for (int u = u0; u < u1 && ok; ++local) {
                const int end = min(u1, (u / p.kb + 1) * p.kb), buf = local & 1;
                if (local >= 2 && !wait_or_abort(acce0 + 8 * buf, ((local >> 1) - 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t dcol = tmem + (uint32_t)(buf * p.mpad);
                for (uint32_t acc = 0; u < end; ++u, acc = 1) {
                    if (!wait_or_abort(full0 + 8 * s, ph, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = a0 + s * sstep, bd = b0 + s * sstep;
                    mma_f16(dcol, ad, bd, idesc, acc);
                    mma_f16(dcol, ad + 2, bd + 2, idesc, 1u);
                    mma_f16(dcol, ad + 4, bd + 4, idesc, 1u);
                    mma_f16(dcol, ad + 6, bd + 6, idesc, 1u);
                    issued = true;
                    mma_commit(empty0 + 8 * s);
                    if (++s == (uint32_t)p.stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (ok) mma_commit(accf0 + 8 * buf);
            }
            if (!ok) raise_abort(abort_flag, p.err);
            if (issued) {
                mma_commit(drain);
                mbar_wait_bounded(drain, 0, kTcWaitNs);
            }
        }
        __syncwarp();
    } else {
        // ---- t, while the weight streams: one rank a warp and step where that fills the warps, else four
        const AdapterArgs &a = p.a;
        const int rk = (int)a.rows * a.rank > 4 * kTWarps * kSms ? 4 : 1, jobs = (int)a.rows * (a.rank / rk);
        for (int j = (warp - 2) * gridDim.x + blockIdx.x; j < jobs; j += kTWarps * gridDim.x) {
            const int m = j / (a.rank / rk), r = j % (a.rank / rk) * rk;
            int raw;
            const int ad = adapter_of_row(a, m, &raw);
            if (ad < 0) continue;  // warp-uniform
            if (rk == 4) shrink_rows<T, 4>(a, p.t, m, r, ad);
            else shrink_rows<T, 1>(a, p.t, m, r, ad);
        }
        // ---- partial sums: lane = channel of the tile, column = row of x
        const int quad = warp & 3;
        int local = 0;
        for (int u = warp < 6 ? u0 : u1; u < u1; ++local) {
            const int tile = u / p.kb, buf = local & 1;
            u = min(u1, (tile + 1) * p.kb);
            if (!wait_or_abort(accf0 + 8 * buf, (local >> 1) & 1, abort_flag)) {
                raise_abort(abort_flag, p.err);
                break;
            }
            tc_fence_after();
            float *dst = p.partial + (long long)(blockIdx.x + tile) * p.mpad * kTN + quad * 32 + lane;
            for (int c = 0; c < p.mpad; c += 16) {
                float v[16];
                tmem_ld16(tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(buf * p.mpad + c), v);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c + i < (int)a.rows) dst[(c + i) * kTN] = v[i];
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acce0 + 8 * buf);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols)
                     : "memory");
    }
}

constexpr int kCombineWarps = 4;

// log2 of the lanes that share a row of B, 8 values each (a power of two)
__host__ __device__ __forceinline__ int lanes_log2(int rank) {
    int l = 0;
    while ((8 << l) < rank) ++l;
    return l;
}
// Channels of a warp: what 8 of its loads cover of B, 256 / 2^l rows, between 16 and a tile.
__host__ __device__ __forceinline__ int channels_of(int rank) { return min(kTN, 256 >> lanes_log2(rank)); }

template <typename T> __global__ void __launch_bounds__(kCombineWarps * 32) adapters_rows_combine(const SmallParams p) {
    __shared__ float term[kCombineWarps][kTN];
    const AdapterArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, m = blockIdx.y;
    const int lw = lanes_log2(a.rank), width = 1 << lw, per = 32 >> lw, cover = channels_of(a.rank);
    const int n0 = (blockIdx.x * kCombineWarps + warp) * cover;
    if (n0 >= p.tiles * kTN) return;  // warp-uniform
    int raw;
    const int ad = adapter_of_row(a, m, &raw);
    if (n0 == 0 && lane == 0) report_bad_adapter(raw, a.adapters, p.err);
    const int chunks = a.rank / 8, c8 = lane & (width - 1), sub = lane >> lw;
    uint4 bv[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i = e * per + sub;
        bv[e] = make_uint4(0, 0, 0, 0);
        if (ad >= 0 && c8 < chunks && i < cover && n0 + i < a.cout)
            bv[e] = ld_nc16(static_cast<const T *>(a.b) + ((long long)ad * a.cout + n0 + i) * a.rank + c8 * 8);
    }
    // the partial sums of the channels' tile, its CTAs in order; lane, lane + 32, ... of the channels
    const int tile = n0 / kTN, total = p.kb * p.tiles, first = run_of(total, tile * p.kb, p.ctas);
    const int last = run_of(total, tile * p.kb + p.kb - 1, p.ctas);
    const float *src = p.partial + ((long long)(first + tile) * p.mpad + m) * kTN + n0 % kTN + lane;
    const T *bias = static_cast<const T *>(a.bias);
    constexpr int kOwn = kTN / 32;
    float y[kOwn], b0[kOwn];
    bool in[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        in[i] = 32 * i + lane < cover && n0 + 32 * i + lane < a.cout;
        b0[i] = bias && in[i] ? to_f32(bias[n0 + 32 * i + lane]) : 0.0f;
        y[i] = 0.0f;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (ad == -2) return;  // warp-uniform
    float4 t0 = make_float4(0.0f, 0.0f, 0.0f, 0.0f), t1 = t0;
    if (ad >= 0 && c8 < chunks) {
        const float4 *tp = reinterpret_cast<const float4 *>(p.t + (long long)m * a.rank + c8 * 8);
        t0 = __ldcg(tp);
        t1 = __ldcg(tp + 1);
    }
#pragma unroll 8
    for (int c = first; c <= last; ++c, src += p.mpad * kTN)
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
            if (in[i]) y[i] += __ldcg(src + 32 * i);
    if (ad >= 0) {
        const float t[8] = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = e * per + sub;
            float f[8], v = 0.0f;
            unpack16<T>(bv[e], f);
#pragma unroll
            for (int k = 0; k < 8; ++k) v = fmaf(f[k], t[k], v);
            if (c8 >= chunks) v = 0.0f;
            for (int s = width >> 1; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
            if (c8 == 0 && i < cover) term[warp][i] = v;
        }
        __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
        if (in[i]) {
            if (ad >= 0) y[i] += term[warp][32 * i + lane];
            static_cast<T *>(a.out)[(long long)m * a.cout + n0 + 32 * i + lane] = from_f32<T>(y[i] + b0[i]);
        }
}

template <typename T>
bool encode(CUtensorMap *m, const void *base, long long cols, long long rows, int box) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t str[1] = {(cuuint64_t)cols * 2};
    const cuuint32_t bx[2] = {(cuuint32_t)kBK, (cuuint32_t)box}, es[2] = {1, 1};
    const CUtensorMapDataType dt = std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                  : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return encode_fn()(m, dt, 2, const_cast<void *>(base), dims, str, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The sizes that follow from the problem alone.
SmallParams plan(const AdapterArgs &a) {
    SmallParams p;
    p.a = a;
    p.mpad = ((int)a.rows + 15) / 16 * 16;
    p.kb = (a.cin + kBK - 1) / kBK;
    p.tiles = (a.cout + kTN - 1) / kTN;
    const long long total = (long long)p.kb * p.tiles;
    // at least two blocks a run: COMBINE reads a partial sum per run
    const long long runs = (total + 1) / 2;
    p.ctas = (int)(runs < kSms ? runs : kSms);
    return p;
}

size_t t_floats(const AdapterArgs &a) { return ((size_t)a.rows * a.rank + 3) / 4 * 4; }

template <typename T> cudaError_t launch_t(const AdapterArgs &a, cudaStream_t stream) {
    const DeviceInfo *dev = device_info();
    if (!encode_fn() || !dev) return cudaErrorNotSupported;
    SmallParams p = plan(a);
    p.t = static_cast<float *>(a.workspace);
    p.partial = p.t + t_floats(a);
    p.err = dev->err;
    p.tmem_cols = 32;
    while (p.tmem_cols < 2 * p.mpad) p.tmem_cols <<= 1;
    // as many stages as fit and as a run has blocks
    const int run = (p.kb * p.tiles + p.ctas - 1) / p.ctas;
    const size_t sbytes = kWBytes + (size_t)p.mpad * kBK * 2, other = 1024 + (2 * kMaxStages + 5) * 8 + 8;
    p.stages = run < 2 ? 2 : run < kMaxStages ? run : kMaxStages;
    while (other + p.stages * sbytes > (size_t)dev->smem_optin) --p.stages;
    const size_t need = other + p.stages * sbytes, share = tensor_memory_share((size_t)dev->smem_optin, p.tmem_cols);
    const size_t smem = need > share ? need : share;
    CUtensorMap wm, xm;
    if (!encode<T>(&wm, a.weight, a.cin, a.cout, kTN) || !encode<T>(&xm, a.x, a.cin, a.rows, p.mpad))
        return cudaErrorInvalidValue;
    static std::atomic<bool> stream_ok[kMaxDev];
    cudaError_t e = allow_smem(adapters_rows_stream<T>, dev->smem_optin, stream_ok);
    if (e != cudaSuccess) return e;
    const int t_ctas = ((int)a.rows * a.rank + kTWarps - 1) / kTWarps;
    const int grid = t_ctas > p.ctas ? (t_ctas < kSms ? t_ctas : kSms) : p.ctas;
    adapters_rows_stream<T><<<grid, kThreads, smem, stream>>>(wm, xm, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const int per_cta = kCombineWarps * channels_of(a.rank);
    cfg.gridDim = dim3((unsigned)((a.cout + per_cta - 1) / per_cta), (unsigned)a.rows);
    cfg.blockDim = dim3(kCombineWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, adapters_rows_combine<T>, p);
}

}  // namespace

size_t adapters_small_workspace(const AdapterArgs &a) {
    const SmallParams p = plan(a);
    return (t_floats(a) + (size_t)(p.ctas + p.tiles) * p.mpad * kTN) * 4;
}

cudaError_t launch_adapters_small(const AdapterArgs &a, cudaStream_t stream) {
    switch (a.dtype) {
        case DType::F16: return launch_t<__half>(a, stream);
        case DType::BF16: return launch_t<__nv_bfloat16>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace dcnb
