// Projection with low-rank adapters of many requests (sm_100a), many rows:
//   t[m, :] = scale[a] * A[a] x[m]             a = adapter of row m's request
//   y[m, n] = bias[n] + sum_k W[n, k] x[m, k] + sum_j B[a][n, j] t[m, j]
// A request owns a range of rows, so a tile of 128 rows meets one request or a
// few.  The adapter term of a tile is therefore nothing but further blocks of
// the same contraction, one set per request in the tile: the tile's rows of t
// against the request's B.  The tensor core adds them to the accumulator that
// already holds x W^T, in the request's rows only: the instruction's mask of
// output lanes leaves the other rows alone (a product with zeros instead would
// carry an infinity of one request's adapter into its neighbours' rows).
//
// Two launches of one kernel.  SHRINK forms t for every pair (tile of 128 rows,
// request in it) and stores the request's rows, scaled and then rounded once
// to the storage type, which the operands of the second product have.  Along
// the rows either the tile or the request advances, so tile + request numbers
// the pairs.  EXPAND runs over the tiles of y, 128 rows x BN channels: the
// blocks of x and W first, then those of t and B.  EXPAND is a programmatic
// dependent of SHRINK and waits for it only before its first load of t.
//
// Both are persistent and warp-specialised: warp 0 streams the 64-wide blocks
// of both operands by TMA (128-byte swizzle, zero fill past every edge) through
// a ring, one thread of warp 1 issues tcgen05.mma into one of two tensor-memory
// accumulators, warps 2..5 read the finished one back, finish it and store.
// Every wait is bounded and gives up when another role has aborted.
#include <cudaTypedefs.h>

#include <type_traits>

#include "dcn_device.h"
#include "dcn_proj_adapters.cuh"
#include "dcn_tcgen05.cuh"

namespace dcnb {
namespace {

constexpr int kBM = 128;
constexpr int kBK = 64;
constexpr int kABytes = kBM * kBK * 2;
constexpr int kThreads = 6 * 32;
constexpr int kMaxStages = 8;
constexpr int kReqCache = 1024;  // requests whose table is kept in shared memory

struct LargeParams {
    int rows, cin, cout, rank, adapters, requests;
    const int32_t *start, *which;
    const float *scale;
    const void *bias;
    void *t;               // [rows, rank]
    void *out;
    int MT, NT;            // tiles of rows, of output channels
    int BN;                // output channels (SHRINK: rank rounded up to 16) of a tile
    int stages, tmem_cols;
    long long jobs;        // tiles of y, or pairs of a tile and a request
    unsigned int *err;
};

// A request's rows inside [0, rows), from the table (in shared or global memory).
struct Requests {
    const int32_t *start, *which;
    int count, rows, adapters;
    __device__ __forceinline__ int at(int s) const { return min(max(start[s], 0), rows); }
    __device__ __forceinline__ int adapter(int s) const { return adapter_of(which, s, adapters); }
    // the first request that ends after row r
    __device__ __forceinline__ int first_ending_after(int r) const {
        int lo = 0, hi = count;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (at(mid + 1) <= r) lo = mid + 1;
            else hi = mid;
        }
        return lo;
    }
    // the request of pair j, -1 if there is none or it has no adapter; its tile is j - request
    __device__ __forceinline__ int of_pair(long long j) const {
        int lo = 0, hi = count;  // the last request whose first pair, at(s) / 128 + s, is at most j
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (at(mid) / kBM + mid <= j) lo = mid + 1;
            else hi = mid;
        }
        const int s = lo - 1;
        if (s < 0) return -1;
        const int tile = (int)(j - s), r0 = at(s), r1 = at(s + 1);
        return r1 > r0 && tile >= r0 / kBM && tile * kBM < r1 && adapter(s) >= 0 ? s : -1;
    }
};

// Bits [lo, hi) of a word; bounds outside [0, 32] are cut off.
__device__ __forceinline__ uint32_t lane_bits(int lo, int hi) {
    lo = max(lo, 0);
    hi = min(hi, 32);
    if (hi <= lo) return 0u;
    return (hi == 32 ? 0xffffffffu : (1u << hi) - 1u) & ~((1u << lo) - 1u);
}

// A product that updates only the accumulator lanes (rows) whose bit in `off` is clear.
__device__ __forceinline__ void mma_f16_lanes(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              const uint32_t *off) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7}, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3])
        : "memory");
}

template <typename T, bool SHRINK>
__global__ void __launch_bounds__(kThreads, 1)
    adapters_gemm_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                         const __grid_constant__ CUtensorMap tmap, const __grid_constant__ CUtensorMap bmap,
                         const LargeParams p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int bbytes = p.BN * kBK * 2, sbytes = kABytes + bbytes;  // BN a multiple of 16: a stage is a multiple of 1 KB
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + p.stages * sbytes);
    // full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * kMaxStages + 5);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int32_t *cache = reinterpret_cast<int32_t *>(tmem_slot + 2);  // [requests + 1] starts, [requests] adapters
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kMaxStages, accf0 = empty0 + 8 * kMaxStages;
    const uint32_t acce0 = accf0 + 16, drain = acce0 + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (SHRINK) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
    const bool cached = p.requests <= kReqCache;
    if (cached) {
        for (int i = threadIdx.x; i <= p.requests; i += kThreads) cache[i] = p.start[i];
        for (int i = threadIdx.x; i < p.requests; i += kThreads) cache[p.requests + 1 + i] = p.which[i];
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
    Requests req;
    req.start = cached ? cache : p.start;
    req.which = cached ? cache + p.requests + 1 : p.which;
    req.count = p.requests;
    req.rows = p.rows;
    req.adapters = p.adapters;
    if (SHRINK && blockIdx.x == 0 && warp >= 2)
        for (int i = threadIdx.x - 64; i < p.requests; i += 128) report_bad_adapter(req.which[i], p.adapters, p.err);
    const int KB = (p.cin + kBK - 1) / kBK, RB = (p.rank + kBK - 1) / kBK;

    if (warp == 0) {
        // ---- producer
        if (lane == 0) {
            uint32_t s = 0, pass = 0;
            long long issued = 0;
            bool ok = true, waited = false;
            auto load = [&](const CUtensorMap *am, int a0, int a1, const CUtensorMap *bm, int b0, int b1) {
                if (pass >= 1 && !wait_or_abort(empty0 + 8 * s, (pass - 1) & 1, abort_flag)) return false;
                mbar_arrive_expect_tx(full0 + 8 * s, (uint32_t)sbytes);
                unsigned char *st = ring + s * sbytes;
                tma_load_2d(smem_u32(st), am, full0 + 8 * s, a0, a1);
                tma_load_2d(smem_u32(st + kABytes), bm, full0 + 8 * s, b0, b1);
                ++issued;
                if (++s == (uint32_t)p.stages) {
                    s = 0;
                    ++pass;
                }
                return true;
            };
            for (long long j = blockIdx.x; j < p.jobs && ok && !*abort_flag; j += gridDim.x) {
                if (SHRINK) {
                    const int r = req.of_pair(j);
                    if (r < 0) continue;
                    const int tile = (int)(j - r), ad = req.adapter(r);
                    for (int kb = 0; kb < KB && ok; ++kb)
                        ok = load(&xmap, kb * kBK, tile * kBM, &wmap, kb * kBK, ad * p.rank);
                } else {
                    const int tile = (int)(j / p.NT), n0 = (int)(j % p.NT) * p.BN;
                    for (int kb = 0; kb < KB && ok; ++kb) ok = load(&xmap, kb * kBK, tile * kBM, &wmap, kb * kBK, n0);
                    if (ok && !waited) {
                        // t comes from the SHRINK kernel: visible from here on, to the TMA too
                        asm volatile("griddepcontrol.wait;" ::: "memory");
                        asm volatile("fence.proxy.async;" ::: "memory");
                        waited = true;
                    }
                    for (int r = req.first_ending_after(tile * kBM); ok && r < p.requests; ++r) {
                        if (req.at(r) >= (tile + 1) * kBM) break;
                        const int ad = req.adapter(r);
                        if (ad < 0 || req.at(r + 1) <= req.at(r)) continue;
                        for (int rb = 0; rb < RB && ok; ++rb)
                            ok = load(&tmap, rb * kBK, tile * kBM, &bmap, rb * kBK, ad * p.cout + n0);
                    }
                }
            }
            if (!ok) raise_abort(abort_flag, p.err);
            // the last load of every stage has landed before the CTA may exit
            for (long long j = issued - 1; j >= 0 && j >= issued - p.stages; --j)
                mbar_wait_bounded(full0 + 8 * (uint32_t)(j % p.stages), (uint32_t)(j / p.stages) & 1, kTcWaitNs);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- one thread issues the products
        if (lane == 0) {
            const int fmt = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
            const uint32_t idesc = instr_desc_f16(fmt, p.BN);
            const uint64_t a0 = smem_desc_sw128(smem_u32(ring)), b0 = smem_desc_sw128(smem_u32(ring + kABytes));
            const uint32_t sstep = (uint32_t)sbytes >> 4;
            uint32_t s = 0, ph = 0;
            int local = 0;
            bool ok = true, issued = false;
            uint32_t dcol = 0, acc = 0;
            // a block of `steps` products of 16 channels each (2 descriptor units), in all rows or
            // outside the lanes `off`
            auto block = [&](int steps, const uint32_t *off) {
                if (!wait_or_abort(full0 + 8 * s, ph, abort_flag)) return false;
                tc_fence_after();
                const uint64_t ad = a0 + s * sstep, bd = b0 + s * sstep;
                if (off) {
                    for (int i = 0; i < steps; ++i) mma_f16_lanes(dcol, ad + 2 * i, bd + 2 * i, idesc, off);
                } else {
                    mma_f16(dcol, ad, bd, idesc, acc);
                    if (steps > 1) mma_f16(dcol, ad + 2, bd + 2, idesc, 1u);
                    if (steps > 2) mma_f16(dcol, ad + 4, bd + 4, idesc, 1u);
                    if (steps > 3) mma_f16(dcol, ad + 6, bd + 6, idesc, 1u);
                }
                acc = 1u;
                issued = true;
                mma_commit(empty0 + 8 * s);
                if (++s == (uint32_t)p.stages) {
                    s = 0;
                    ph ^= 1u;
                }
                return true;
            };
            for (long long j = blockIdx.x; j < p.jobs && ok; j += gridDim.x) {
                if (SHRINK && req.of_pair(j) < 0) continue;
                const int buf = local & 1;
                if (local >= 2 && !wait_or_abort(acce0 + 8 * buf, ((local >> 1) - 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                dcol = tmem + (uint32_t)(buf * p.BN);
                acc = 0;
                for (int kb = 0; kb < KB && ok; ++kb) ok = block(min(4, (p.cin - kb * kBK + 15) / 16), nullptr);
                if (!SHRINK) {
                    const int tile = (int)(j / p.NT);
                    for (int r = req.first_ending_after(tile * kBM); ok && r < p.requests; ++r) {
                        if (req.at(r) >= (tile + 1) * kBM) break;
                        if (req.adapter(r) < 0 || req.at(r + 1) <= req.at(r)) continue;
                        const int r0 = max(req.at(r) - tile * kBM, 0), r1 = min(req.at(r + 1) - tile * kBM, kBM);
                        uint32_t off[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) off[i] = ~lane_bits(r0 - 32 * i, r1 - 32 * i);
                        for (int rb = 0; rb < RB && ok; ++rb) ok = block(min(4, (p.rank - rb * kBK + 15) / 16), off);
                    }
                }
                if (!ok) break;
                mma_commit(accf0 + 8 * buf);
                ++local;
            }
            if (!ok) raise_abort(abort_flag, p.err);
            if (issued) {
                // every product has finished before tensor memory is freed
                mma_commit(drain);
                mbar_wait_bounded(drain, 0, kTcWaitNs);
            }
        }
        __syncwarp();
    } else {
        // ---- epilogue: warp w reads tensor-memory lanes 32 * (w % 4) .. +31 = rows of the tile
        const int quad = warp & 3;
        const T *bias = static_cast<const T *>(p.bias);
        const int covered0 = p.requests ? req.at(0) : 0, covered1 = p.requests ? req.at(p.requests) : 0;
        int local = 0;
        for (long long j = blockIdx.x; j < p.jobs; j += gridDim.x) {
            int r = 0, row, n0, ncols;
            T *dst;
            float mul = 1.0f;
            bool write;
            if (SHRINK) {
                r = req.of_pair(j);
                if (r < 0) continue;
                row = (int)(j - r) * kBM + quad * 32 + lane;
                n0 = 0;
                ncols = p.rank;
                dst = static_cast<T *>(p.t) + (long long)row * p.rank;
                mul = p.scale ? p.scale[req.adapter(r)] : 1.0f;
                write = row >= req.at(r) && row < req.at(r + 1);
            } else {
                row = (int)(j / p.NT) * kBM + quad * 32 + lane;
                n0 = (int)(j % p.NT) * p.BN;
                ncols = min(p.BN, p.cout - n0);
                dst = static_cast<T *>(p.out) + (long long)row * p.cout + n0;
                write = row >= covered0 && row < covered1;
            }
            const int buf = local & 1;
            if (!wait_or_abort(accf0 + 8 * buf, (local >> 1) & 1, abort_flag)) {
                raise_abort(abort_flag, p.err);
                break;
            }
            tc_fence_after();
            for (int c = 0; c < ncols; c += 16) {  // warp-uniform
                float v[16];
                tmem_ld16(tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(buf * p.BN + c), v);
                if (SHRINK) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] *= mul;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (c + 8 * h >= ncols) continue;  // cout and rank are multiples of 8
                    if (!SHRINK && bias) {
                        float b[8];
                        unpack16<T>(ld_nc16(bias + n0 + c + 8 * h), b);
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[8 * h + i] += b[i];
                    }
                    if (write) *reinterpret_cast<uint4 *>(dst + c + 8 * h) = pack16<T>(v + 8 * h);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acce0 + 8 * buf);
            ++local;
        }
    }
    // a CTA that had no tile to load t for still outlives the SHRINK kernel: the call's next user of the
    // workspace is ordered behind this kernel
    if (!SHRINK) asm volatile("griddepcontrol.wait;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols)
                     : "memory");
    }
}

// 64-column boxes of `box` rows over a [rows, cols] matrix of T.
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

long long pairs_of(const AdapterArgs &a) { return (a.rows + kBM - 1) / kBM + a.requests; }

int tmem_columns(int bn) {
    int cols = 32;
    while (cols < 2 * bn) cols <<= 1;
    return cols;
}

size_t smem_bytes(int stages, int bn, int requests) {
    return 1024 + (size_t)stages * (kABytes + bn * kBK * 2) + (2 * kMaxStages + 5) * 8 + 8 +
           (requests <= kReqCache ? (size_t)(2 * requests + 1) * 4 : 0);
}

template <typename T, bool SHRINK>
cudaError_t launch_gemm(LargeParams &p, const DeviceInfo *dev, const CUtensorMap &x, const CUtensorMap &w,
                        const CUtensorMap &t, const CUtensorMap &b, cudaStream_t stream) {
    p.tmem_cols = tmem_columns(p.BN);
    int stages = kMaxStages;
    while (stages > 2 && smem_bytes(stages, p.BN, p.requests) > (size_t)dev->smem_optin) --stages;
    p.stages = stages;
    const size_t smem = smem_bytes(stages, p.BN, p.requests);
    auto kern = adapters_gemm_kernel<T, SHRINK>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.jobs < dev->sms ? p.jobs : dev->sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = SHRINK ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, kern, x, w, t, b, p);
}

template <typename T> cudaError_t launch_t(const AdapterArgs &a, cudaStream_t stream) {
    const DeviceInfo *dev = device_info();
    if (!encode_fn() || !dev) return cudaErrorNotSupported;
    LargeParams p;
    p.rows = (int)a.rows;
    p.cin = a.cin; p.cout = a.cout; p.rank = a.rank; p.adapters = a.adapters; p.requests = a.requests;
    p.start = a.start; p.which = a.which; p.scale = a.scale; p.bias = a.bias;
    p.t = a.workspace;
    p.out = a.out;
    p.err = dev->err;
    p.MT = (int)((a.rows + kBM - 1) / kBM);
    const long long pairs = pairs_of(a);

    CUtensorMap xm, am, wm, tm, bm;
    const int rank16 = (a.rank + 15) / 16 * 16;
    // the tile width whose rounds of tiles over the SMs cost least: a tile costs its columns, plus a
    // constant share (the rows of x it streams and its epilogue) of 48 columns
    int bn = 0;
    long long best = 0;
    for (int c = 256; c >= 64; c /= 2) {
        const long long tiles = (long long)p.MT * ((a.cout + c - 1) / c);
        const long long cost = (tiles + dev->sms - 1) / dev->sms * (c + 48);
        if (!bn || cost < best) {
            bn = c;
            best = cost;
        }
    }
    if (!encode<T>(&xm, a.x, a.cin, a.rows, kBM) || !encode<T>(&wm, a.weight, a.cin, a.cout, bn) ||
        !encode<T>(&tm, a.workspace, a.rank, a.rows, kBM))
        return cudaErrorInvalidValue;
    am = bm = wm;  // never read without adapters
    if (a.adapters > 0 && (!encode<T>(&am, a.a, a.cin, (long long)a.adapters * a.rank, rank16) ||
                           !encode<T>(&bm, a.b, a.rank, (long long)a.adapters * a.cout, bn)))
        return cudaErrorInvalidValue;
    p.BN = rank16;
    p.NT = 1;
    p.jobs = pairs;
    cudaError_t e = launch_gemm<T, true>(p, dev, xm, am, xm, am, stream);
    if (e != cudaSuccess) return e;
    p.BN = bn;
    p.NT = (a.cout + bn - 1) / bn;
    p.jobs = (long long)p.MT * p.NT;
    return launch_gemm<T, false>(p, dev, xm, wm, tm, bm, stream);
}

}  // namespace

size_t adapters_large_workspace(const AdapterArgs &a) { return (size_t)a.rows * a.rank * 2; }

cudaError_t launch_adapters_large(const AdapterArgs &a, cudaStream_t stream) {
    switch (a.dtype) {
        case DType::F16: return launch_t<__half>(a, stream);
        case DType::BF16: return launch_t<__nv_bfloat16>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

// Few rows are bound by the weight's bytes and take the row-wise kernels.
size_t proj_adapters_workspace(const AdapterArgs &a) {
    return a.rows <= kMaxSmallRows ? adapters_small_workspace(a) : adapters_large_workspace(a);
}

cudaError_t launch_proj_adapters(const AdapterArgs &a, cudaStream_t stream) {
    return a.rows <= kMaxSmallRows ? launch_adapters_small(a, stream) : launch_adapters_large(a, stream);
}

}  // namespace dcnb
