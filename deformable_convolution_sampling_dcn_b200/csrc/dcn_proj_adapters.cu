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
// SHRINK forms t for every pair (tile of 128 rows, request in it) and stores
// the request's rows, scaled.  The operands of the second product have the
// storage type, so t is held in 32 bits as the sum of two values of it, t rounded
// and the rest rounded (22 bits of mantissa in fp16, 16 in bf16, against 11 and 8
// of one value: bf16 16111 rows 2048 -> 2048, rank 64, the error against 64 bits
// 1.84e-3 with one value, 1.66e-3 with two, which is the output's own rounding).
// fp16 has no room above 65504: eight neighbours of a row of t that go beyond 2^15
// are scaled down by a power of two, whose exponent is kept, and EXPAND adds what is
// missing in fp32 when it finishes the row.  Along the rows either the tile or the
// request advances, so tile + request numbers the pairs.
//
// EXPAND runs over the tiles of y: the blocks of x and W first, then those of t
// and B.  A tile is 256 rows x BN channels by a pair of CTAs (cta_group::2):
// each CTA stages its own 128 rows and half of the channels, 64 KB by both for
// 256 x 256 x 64 products (single CTAs with 128 x 256 tiles stage 96 KB for as many,
// and took 138 us where pairs took 122).  EXPAND is a programmatic dependent of
// SHRINK and waits for it before its first load of t and, in fp16, of the exponents.
//
// The two values of t take twice the least workspace of a call.  With less than
// that the rows go in several passes, two launches each, with t of one pass at a
// time.
//
// Where the tiles are fewer than the SMs, a cluster of CTAs (SHRINK) or of pairs
// (EXPAND) splits the contraction of one tile; the parts meet in distributed
// shared memory and are added in the order of the splits, each CTA finishing a
// share of the columns.
//
// Both are persistent and warp-specialised: warp 0 streams the 64-wide blocks
// of both operands by TMA (128-byte swizzle, zero fill past every edge) through
// a ring, one thread of warp 1 (of the pair's first CTA) issues tcgen05.mma into
// one of two tensor-memory accumulators, the others (four warps in SHRINK, eight in
// EXPAND) read the finished one back, finish it and store.  Every wait is bounded
// and gives up when another role of the CTA has aborted.
//
// Measured (one B200): fp16 12800 rows 512 -> 512, rank 16 21.6 us (330 TFLOP/s,
// bound by the chain of latencies of the two launches; the tensor pipe is busy for
// a fifth of EXPAND); bf16 16111 rows 2048 -> 2048, rank 64 127 us (1.1 PFLOP/s), 97
// us of it the products with W, the tensor pipe busy for 71 % of EXPAND and L2 at 40 %
// of its rate.  With t rounded to one value they took 21.1 and 120 us.  Every request
// in a tile is a set of blocks of its own: 512 single tokens 1024 -> 4096 246 us.
#include <cudaTypedefs.h>

#include <type_traits>

#include "dcn_device.h"
#include "dcn_proj_adapters.cuh"
#include "dcn_tcgen05.cuh"

namespace dcnb {
namespace {

constexpr int kBM = 128;                 // rows of a CTA
constexpr int kBK = 64;
constexpr int kABytes = kBM * kBK * 2;
constexpr int kThreads = 6 * 32;
constexpr int kMaxStages = 8;
// CTA pairs of split tiles.  A cluster lies within one of the GPU's processing clusters, and some of 64 pairs in
// clusters of eight CTAs waited for the others to end (80 rows 1024 -> 1024: 30 us against 17 without splits).
constexpr int kClusterPairs = 32;
constexpr int kReqCache = 1024;  // requests whose table is kept in shared memory

struct LargeParams {
    int rows, cin, cout, rank, adapters, requests;
    const int32_t *start, *which;
    const float *scale;
    const void *bias;
    // this pass: rows row0 .. row0 + rows - 1 of the request table, t [2, rows, rank] and (fp16) the exponents of its
    // groups of eight ranks [rows, 16], both for rows with an adapter only; out starts at row0
    int row0;
    void *t;
    unsigned char *shift;
    const void *b;
    void *out;
    int NT;                // EXPAND: tiles of output channels
    int BN;                // EXPAND: output channels of a tile; SHRINK: rank rounded up to 16
    int stages, tmem_cols;
    int aw;                // bytes of a row of an adapter block: 32, 64 or 128, its swizzle too
    int splits;            // of the contraction; a cluster has one job where this is not 1
    long long jobs;        // EXPAND: tiles of y; SHRINK: pairs of a tile and a request, empty requests included
    unsigned int *err;
};

// A request's rows inside [0, rows) of this pass, from the table (in shared or global memory).
struct Requests {
    const int32_t *start, *which;
    int count, row0, rows, adapters;
    __device__ __forceinline__ int at(int s) const { return min(max(start[s], row0) - row0, rows); }
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
    // Leaves out the empty requests at the end, with which a program fills its table up to a fixed size.  By all threads,
    // once the table is there.
    __device__ __forceinline__ void drop_empty_tail() {
        const int end = at(count);
        if (at(count - 1) < end) return;
        const Requests all = *this;
        count = warp_first(count, [&](int s) { return all.at(s) >= end; });
    }
};

// The requests that own rows of [r0, r1), which are at most as many as the rows (a table that is not ascending ends
// there); empty ones between them are passed over by search.
struct RequestsOf {
    const Requests &q;
    int r, lo, hi;  // request r, and its rows lo .. hi - 1
    int r1, left;
    __device__ __forceinline__ RequestsOf(const Requests &q_, int r0, int r1_) : q(q_), r1(r1_), left(r1_ - r0) {
        go(q.first_ending_after(r0));
    }
    __device__ __forceinline__ bool valid() const { return left > 0 && r < q.count && lo < r1; }
    __device__ __forceinline__ void next() {
        --left;
        if (++r >= q.count) return;
        lo = hi;
        hi = q.at(r + 1);
        if (hi <= lo) go(max(r, q.first_ending_after(lo)));
    }
    __device__ __forceinline__ void go(int to) {
        r = to;
        if (r >= q.count) return;
        lo = q.at(r);
        hi = q.at(r + 1);
    }
};

// Shared memory of a CTA: the ring, the barriers, the tensor-memory address, the abort flag and the request
// table.
struct Smem {
    unsigned char *ring;
    uint32_t full, empty, acc_full, acc_empty, drain;  // barriers: kMaxStages, kMaxStages, 2, 2, 1
    uint32_t *tmem_slot;
    volatile int *abort_flag;
    int32_t *cache;  // [requests + 1] starts, [requests] adapters
    __device__ __forceinline__ Smem(unsigned char *raw, int ring_bytes) {
        ring = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
        uint64_t *bars = reinterpret_cast<uint64_t *>(ring + ring_bytes);
        full = smem_u32(bars);
        empty = full + 8 * kMaxStages;
        acc_full = empty + 8 * kMaxStages;
        acc_empty = acc_full + 16;
        drain = acc_empty + 16;
        tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * kMaxStages + 5);
        abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
        cache = reinterpret_cast<int32_t *>(tmem_slot + 2);
    }
    // by one thread; `readers` warps empty an accumulator
    __device__ __forceinline__ void init(int readers) const {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, readers);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    // by all threads, before a CTA barrier
    __device__ __forceinline__ Requests requests(const LargeParams &p) const {
        Requests r;
        const bool cached = p.requests <= kReqCache;
        if (cached) {
            for (int i = threadIdx.x; i <= p.requests; i += blockDim.x) cache[i] = p.start[i];
            for (int i = threadIdx.x; i < p.requests; i += blockDim.x) cache[p.requests + 1 + i] = p.which[i];
        }
        r.start = cached ? cache : p.start;
        r.which = cached ? cache + p.requests + 1 : p.which;
        r.count = p.requests;
        r.row0 = p.row0;
        r.rows = p.rows;
        r.adapters = p.adapters;
        return r;
    }
};

// Position in the ring.
struct Slot {
    uint32_t s = 0, pass = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++s == (uint32_t)stages) {
            s = 0;
            ++pass;
        }
    }
};

__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of CTA `rank`'s variable that is at `addr` in this one.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float load_remote(uint32_t cluster_addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr));
    return v;
}

// A split's accumulator, 128 rows (this warp's 32, one a lane) x `cols`, into its shared memory, column by column.
__device__ __forceinline__ void dump_accumulator(uint32_t taddr, float *dst, int cols, int first, int step) {
    for (int c = first; c < cols; c += step) {
        float v[16];
        tmem_ld16(taddr + (uint32_t)c, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) dst[(c + i) * 128] = v[i];
    }
}
// Sum of the splits' values of 8 columns from c on, in the order of the splits; their CTAs are `stride` ranks apart.
__device__ __forceinline__ void add_splits(uint32_t addr, int c, int splits, int first_rank, int stride, float *v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    for (int s = 0; s < splits; ++s) {
        const uint32_t base = in_cta(addr + (uint32_t)(c * 128 * 4), first_rank + s * stride);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += load_remote(base + (uint32_t)(i * 128 * 4));
    }
}
__device__ __forceinline__ void arrive_remote(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

constexpr int kShiftBytes = 16;  // of a row: the exponents of its (up to) 128 / 8 groups

// Eight values of t as two of the storage type each, the second of which is the first one's rounding error: exact in
// fp32, then rounded.  Infinities and NaN are the first value alone.  Returns the exponent of the power of two by which
// the values are divided, so that the largest finite one stays below 2^15 in fp16; in [0, 113].
template <typename T> __device__ __forceinline__ uint32_t store_t(T *first, T *second, float *v) {
    const float inf = __int_as_float(0x7f800000);
    uint32_t shift = 0;
    if constexpr (std::is_same<T, __half>::value) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fabsf(v[i]) < inf ? fmaxf(m, fabsf(v[i])) : m;
        shift = (uint32_t)max((int)(__float_as_uint(m) >> 23) - 127 - 14, 0);
        const float down = __uint_as_float((127 - shift) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= down;
    } else {
        // a finite value past the largest of bf16 does not round up to an infinity
        const float top = __uint_as_float(0x7f7f0000u);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (fabsf(v[i]) < inf) v[i] = fminf(fmaxf(v[i], -top), top);
    }
    const uint4 hi = pack16<T>(v);
    float f[8];
    unpack16<T>(hi, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fabsf(f[i]) < inf ? v[i] - f[i] : 0.0f;
    *reinterpret_cast<uint4 *>(first) = hi;
    *reinterpret_cast<uint4 *>(second) = pack16<T>(f);
    return shift;
}

// What the product with a row of t leaves out for one channel: (2^shift - 1) b . t over the groups with a shift.
template <typename T>
__device__ __noinline__ float missing_term(const T *b, const T *first, const T *second, const unsigned char *shift,
                                           int rank) {
    float sum = 0.0f;
    for (int k = 0; k < rank; k += 8) {
        const uint32_t e = __ldcg(shift + k / 8);
        if (e == 0) continue;
        const float mul = __uint_as_float((127 + e) << 23) - 1.0f;
        float f[8], t0[8], t1[8];
        unpack16<T>(ld_nc16(b + k), f);
        unpack16<T>(__ldcg(reinterpret_cast<const uint4 *>(first + k)), t0);
        unpack16<T>(__ldcg(reinterpret_cast<const uint4 *>(second + k)), t1);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(f[i], (t0[i] + t1[i]) * mul, sum);
    }
    return sum;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    adapters_shrink_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap amap,
                           const LargeParams p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    constexpr bool kShifted = std::is_same<T, __half>::value;
    const int sbytes = kABytes + p.BN * kBK * 2;  // BN a multiple of 16: a stage is a multiple of 1 KB
    const Smem sm(smem_raw, p.stages * sbytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) sm.init(4);
    Requests req = sm.requests(p);
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(sm.tmem_slot)),
                     "r"(p.tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *sm.tmem_slot;
    // not before this CTA has its columns: EXPAND holds its own while it waits for all of SHRINK
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    req.drop_empty_tail();
    if (blockIdx.x == 0 && warp >= 2)
        for (int i = threadIdx.x - 64; i < req.count; i += 128)
            if (req.at(i + 1) > req.at(i)) report_bad_adapter(req.which[i], p.adapters, p.err);
    const int blocks = (p.cin + kBK - 1) / kBK;
    // this CTA's part of the contraction and its cluster's job
    const int split = p.splits > 1 ? (int)cta_rank() : 0;
    const int kb0 = blocks * split / p.splits, kb1 = blocks * (split + 1) / p.splits;
    const long long job0 = blockIdx.x / p.splits, jobs_step = gridDim.x / p.splits;
    const long long jobs = (p.rows + kBM - 1) / kBM + req.count;  // pairs of a tile and a request: at most the launch's

    if (warp == 0) {
        // ---- producer
        if (lane == 0) {
            Slot at;
            long long issued = 0;
            bool ok = true;
            for (long long j = job0; j < jobs && ok; j += jobs_step) {
                const int r = req.of_pair(j);
                if (r < 0) continue;
                const int row = (int)(j - r) * kBM, arow = req.adapter(r) * p.rank;
                for (int kb = kb0; kb < kb1; ++kb) {
                    const uint32_t full = sm.full + 8 * at.s;
                    if (at.pass >= 1 && !wait_or_abort(sm.empty + 8 * at.s, (at.pass - 1) & 1, sm.abort_flag)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(full, (uint32_t)sbytes);
                    const uint32_t st = smem_u32(sm.ring) + at.s * sbytes;
                    tma_load_2d(st, &xmap, full, kb * kBK, row);
                    tma_load_2d(st + kABytes, &amap, full, kb * kBK, arow);
                    ++issued;
                    at.next(p.stages);
                }
            }
            if (!ok) raise_abort(sm.abort_flag, p.err);
            // the last load of every stage has landed before the CTA may exit
            for (long long j = issued - 1; j >= 0 && j >= issued - p.stages; --j)
                mbar_wait_bounded(sm.full + 8 * (uint32_t)(j % p.stages), (uint32_t)(j / p.stages) & 1, kTcWaitNs);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- one thread issues the products
        if (lane == 0) {
            const uint32_t idesc = instr_desc_f16(std::is_same<T, __nv_bfloat16>::value ? 1 : 0, p.BN);
            const uint64_t a0 = smem_desc_sw128(smem_u32(sm.ring)), b0 = smem_desc_sw128(smem_u32(sm.ring + kABytes));
            const uint32_t sstep = (uint32_t)sbytes >> 4;
            Slot at;
            int local = 0;
            bool ok = true, issued = false;
            for (long long j = job0; j < jobs && ok; j += jobs_step) {
                if (req.of_pair(j) < 0) continue;
                const int buf = local & 1;
                if (local >= 2 && !wait_or_abort(sm.acc_empty + 8 * buf, ((local >> 1) - 1) & 1, sm.abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t dcol = tmem + (uint32_t)(buf * p.BN);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!wait_or_abort(sm.full + 8 * at.s, at.pass & 1, sm.abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = a0 + at.s * sstep, bd = b0 + at.s * sstep;
                    // steps of 16 elements = 2 descriptor units; columns past cin are zeros
                    mma_f16(dcol, ad, bd, idesc, kb != kb0);
                    mma_f16(dcol, ad + 2, bd + 2, idesc, 1u);
                    mma_f16(dcol, ad + 4, bd + 4, idesc, 1u);
                    mma_f16(dcol, ad + 6, bd + 6, idesc, 1u);
                    issued = true;
                    mma_commit(sm.empty + 8 * at.s);
                    at.next(p.stages);
                }
                if (!ok) break;
                mma_commit(sm.acc_full + 8 * buf);
                ++local;
            }
            if (!ok) raise_abort(sm.abort_flag, p.err);
            if (issued) {
                // every product has finished before tensor memory is freed
                mma_commit(sm.drain);
                mbar_wait_bounded(sm.drain, 0, kTcWaitNs);
            }
        }
        __syncwarp();
    } else {
        // ---- epilogue: warp w reads tensor-memory lanes 32 * (w % 4) .. +31 = rows of the tile
        const int quad = warp & 3;
        int local = 0;
        for (long long j = job0; j < jobs; j += jobs_step) {
            const int r = req.of_pair(j);
            if (r < 0) continue;
            const int row = (int)(j - r) * kBM + quad * 32 + lane, buf = local & 1;
            const bool mine = row >= req.at(r) && row < req.at(r + 1);
            const float mul = p.scale ? p.scale[req.adapter(r)] : 1.0f;
            T *dst = static_cast<T *>(p.t) + (long long)row * p.rank, *rest = dst + (long long)p.rows * p.rank;
            if (!wait_or_abort(sm.acc_full + 8 * buf, (local >> 1) & 1, sm.abort_flag)) {
                raise_abort(sm.abort_flag, p.err);
                break;
            }
            tc_fence_after();
            if (p.splits > 1) {
                // the products have read the ring
                dump_accumulator(tmem + ((uint32_t)(32 * quad) << 16), reinterpret_cast<float *>(sm.ring) + quad * 32 + lane,
                                 p.BN, 0, 16);
                break;
            }
            const uint32_t acc = tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(buf * p.BN);
            for (int c = 0; c < p.rank; c += 16) {  // warp-uniform
                float v[16];
                tmem_ld16(acc + (uint32_t)c, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] *= mul;
                if (mine) {
                    uint32_t shift = store_t<T>(dst + c, rest + c, v);
                    if (c + 8 < p.rank) shift |= store_t<T>(dst + c + 8, rest + c + 8, v + 8) << 8;
                    if (kShifted)
                        *reinterpret_cast<uint16_t *>(p.shift + (long long)row * kShiftBytes + c / 8) = (uint16_t)shift;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sm.acc_empty + 8 * buf);
            ++local;
        }
    }
    if (p.splits > 1) {
        __syncwarp();
        cluster_sync();
        const int r = req.of_pair(job0), quad = warp & 3;
        if (r >= 0 && warp >= 2) {
            const int row = (int)(job0 - r) * kBM + quad * 32 + lane;
            const float mul = p.scale ? p.scale[req.adapter(r)] : 1.0f;
            const uint32_t addr = smem_u32(sm.ring) + (uint32_t)(quad * 32 + lane) * 4;
            T *dst = static_cast<T *>(p.t) + (long long)row * p.rank, *rest = dst + (long long)p.rows * p.rank;
            for (int c = 8 * split; c < p.rank; c += 8 * p.splits) {
                float v[8];
                add_splits(addr, c, p.splits, 0, 1, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= mul;
                if (row >= req.at(r) && row < req.at(r + 1)) {
                    const uint32_t shift = store_t<T>(dst + c, rest + c, v);
                    if (kShifted) p.shift[(long long)row * kShiftBytes + c / 8] = (unsigned char)shift;
                }
            }
        }
        __syncwarp();
        cluster_sync();  // the other CTAs may still read this one's sums
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols)
                     : "memory");
    }
}

// ---- CTA pairs

// Fetches a tensor map ahead of its first use.
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// Load into this CTA's shared memory that completes on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1,
                                                 int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
// Brings a box to L2.
__device__ __forceinline__ void prefetch_2d(const CUtensorMap *map, int c0, int c1) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(c0), "r"(c1)
                 : "memory");
}
// 256 rows: the first CTA's 128 and the second's; N columns, half of the operand in each CTA.
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// The same, adding only to the accumulator rows whose bit in `off` is clear.
__device__ __forceinline__ void mma_pair_rows(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              const uint32_t *off) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7, %8, %9, %10, %11}, p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3]), "r"(off[4]),
        "r"(off[5]), "r"(off[6]), "r"(off[7])
        : "memory");
}
// Arrive on `bar` of both CTAs of the pair (ranks `leader` and the next) once every product this thread issued so far
// is complete.
__device__ __forceinline__ void commit_pair(uint32_t bar, int leader) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)(3 << leader))
        : "memory");
}

// Box of 64 columns x 32 rows from shared memory (128-byte swizzle); completes in this thread's bulk groups.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, uint32_t src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map), "r"(src),
                 "r"(c0), "r"(c1)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// Bits [lo, hi) of a word; bounds outside [0, 32] are cut off.
__device__ __forceinline__ uint32_t lane_bits(int lo, int hi) {
    lo = max(lo, 0);
    hi = min(hi, 32);
    if (hi <= lo) return 0u;
    return (hi == 32 ? 0xffffffffu : (1u << hi) - 1u) & ~((1u << lo) - 1u);
}

// The descriptor of a 128-byte-swizzled operand for one of 32- or 64-byte rows in the swizzle of that width: 8-row
// groups 256 or 512 bytes apart.
__device__ __forceinline__ uint64_t narrow_desc(uint64_t d, int row_bytes) {
    if (row_bytes == 128) return d;
    d &= ~((7ull << 61) | (0x3fffull << 32));
    return d | (uint64_t)(row_bytes == 64 ? 4 : 6) << 61 | (uint64_t)(8 * row_bytes >> 4) << 32;
}

constexpr int kPairRows = 2 * kBM;
constexpr int kOutBytes = 32 * kBK * 2;           // a warp's staged box of y
constexpr int kExpandThreads = 10 * 32;            // eight epilogue warps
constexpr int kOutStage = 8 * kOutBytes + 8 * kBK * 4;  // and the bias of a chunk in fp32, for each of them

template <typename T>
__global__ void __launch_bounds__(kExpandThreads, 1)
    adapters_expand_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                           const __grid_constant__ CUtensorMap tmap, const __grid_constant__ CUtensorMap bmap,
                           const __grid_constant__ CUtensorMap ymap, const LargeParams p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    constexpr bool kShifted = std::is_same<T, __half>::value;
    const int sbytes = kABytes + p.BN / 2 * kBK * 2;
    const Smem sm(smem_raw, p.stages * sbytes + kOutStage);  // the staged boxes of y follow the ring
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = (int)cta_rank(), rank = crank & 1, split = crank >> 1, leader = crank & ~1;
    const long long pair0 = blockIdx.x / (2 * p.splits), pairs = gridDim.x / (2 * p.splits);
    if (threadIdx.x == 0) {
        sm.init(16);  // the epilogue warps of both CTAs
        prefetch_map(&xmap);
        prefetch_map(&wmap);
        prefetch_map(&tmap);
        prefetch_map(&bmap);
        prefetch_map(&ymap);
    }
    Requests req = sm.requests(p);
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(sm.tmem_slot)),
                     "r"(p.tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the other CTA's barriers and tensor memory are ready
    tc_fence_after();
    const uint32_t tmem = *sm.tmem_slot;
    req.drop_empty_tail();
    const int blocks = (p.cin + kBK - 1) / kBK, RB = (p.rank + kBK - 1) / kBK;
    // this pair's part of the contraction; the adapters' blocks belong to the last one
    const int kb0 = blocks * split / p.splits, kb1 = blocks * (split + 1) / p.splits;
    const bool adapters = split == p.splits - 1;
    // values of t that a stage holds: both where their rows of aw bytes fit the place of the 128-byte rows of x
    const int held = p.aw < 128 ? 2 : 1;
    // The adapter of a row of some request whose t has an exponent other than 0, else -1.  The exponents are written for
    // rows with an adapter only: whether a row has one is asked where they are not zero.
    auto shifted_row = [&](int row, bool covered) {
        if (!kShifted || !p.shift || !covered) return -1;
        const uint4 e = __ldcg(reinterpret_cast<const uint4 *>(p.shift + (long long)row * kShiftBytes));
        const uint32_t w[4] = {e.x, e.y, e.z, e.w};
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int bytes = p.rank / 8 - 4 * i;  // of the word that belong to the rank
            if (bytes > 0) any |= bytes >= 4 ? w[i] : w[i] & ((1u << (8 * bytes)) - 1);
        }
        if (any == 0) return -1;
        const int r = req.first_ending_after(row);
        return r < req.count && req.at(r) <= row ? req.adapter(r) : -1;
    };
    auto missing = [&](int row, int ad, int channel) {
        const T *t = static_cast<const T *>(p.t) + (long long)row * p.rank;
        return missing_term<T>(static_cast<const T *>(p.b) + ((long long)ad * p.cout + channel) * p.rank, t,
                               t + (long long)p.rows * p.rank, p.shift + (long long)row * kShiftBytes, p.rank);
    };

    if (warp == 0) {
        // ---- producer: this CTA's rows and half of the channels; both CTAs' loads complete on the first one's
        // barrier, which expects the bytes of both
        if (lane == 0) {
            Slot at;
            long long issued = 0;
            bool ok = true, waited = false;
            const uint32_t full0 = in_cta(sm.full, leader);
            // the blocks at column k: `value` below 0 of x and W, else of t, from that value of it on, and B
            auto load = [&](int value, int k, int row, int brow, uint32_t bytes) {
                if (at.pass >= 1 && !wait_or_abort(sm.empty + 8 * at.s, (at.pass - 1) & 1, sm.abort_flag)) return false;
                if (rank == 0) mbar_arrive_expect_tx(sm.full + 8 * at.s, 2 * bytes);
                const uint32_t st = smem_u32(sm.ring) + at.s * sbytes;
                if (value < 0) tma_load_2d_pair(st, &xmap, full0 + 8 * at.s, k, row);
                else tma_load_3d_pair(st, &tmap, full0 + 8 * at.s, k, row, value);
                tma_load_2d_pair(st + kABytes, value < 0 ? &wmap : &bmap, full0 + 8 * at.s, k, brow);
                ++issued;
                at.next(p.stages);
                return true;
            };
            for (long long j = pair0; j < p.jobs && ok; j += pairs) {
                const int tile = (int)(j / p.NT) * kPairRows, row = tile + rank * kBM;
                const int n0 = (int)(j % p.NT) * p.BN + rank * (p.BN / 2);
                for (int kb = kb0; kb < kb1 && ok; ++kb) ok = load(-1, kb * kBK, row, n0, sbytes);
                if (!adapters) continue;
                if (ok && !waited) {
                    // the first tile's B, which does not depend on SHRINK, comes to L2 meanwhile
                    for (RequestsOf w(req, tile, tile + kPairRows); w.valid(); w.next())
                        if (w.hi > w.lo && req.adapter(w.r) >= 0)
                            for (int rb = 0; rb < RB; ++rb) prefetch_2d(&bmap, rb * kBK, req.adapter(w.r) * p.cout + n0);
                    // t comes from the SHRINK kernel: visible from here on, to the TMA too
                    asm volatile("griddepcontrol.wait;" ::: "memory");
                    asm volatile("fence.proxy.async;" ::: "memory");
                    waited = true;
                }
                for (RequestsOf w(req, tile, tile + kPairRows); ok && w.valid(); w.next()) {
                    const int ad = req.adapter(w.r);
                    if (ad < 0 || w.hi <= w.lo) continue;
                    for (int rb = 0; rb < RB && ok; ++rb)
                        for (int v = 0; v < 2 && ok; v += held)
                            ok = load(v, rb * kBK, row, ad * p.cout + n0, (held * kBM + p.BN / 2) * p.aw);
                }
            }
            if (!ok) raise_abort(sm.abort_flag, p.err);
            // the last loads of every stage, of both CTAs, have landed before the pair may exit
            if (rank == 0)
                for (long long j = issued - 1; j >= 0 && j >= issued - p.stages; --j)
                    mbar_wait_bounded(sm.full + 8 * (uint32_t)(j % p.stages), (uint32_t)(j / p.stages) & 1, kTcWaitNs);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- one thread of the first CTA issues the products
        if (rank == 0 && lane == 0) {
            const uint32_t idesc = (instr_desc_f16(std::is_same<T, __nv_bfloat16>::value ? 1 : 0, p.BN) &
                                    ~(31u << 24)) | ((uint32_t)(kPairRows >> 4) << 24);
            const uint64_t a0 = smem_desc_sw128(smem_u32(sm.ring)), b0 = smem_desc_sw128(smem_u32(sm.ring + kABytes));
            const uint64_t a1 = narrow_desc(a0, p.aw), b1 = narrow_desc(b0, p.aw);
            const uint32_t sstep = (uint32_t)sbytes >> 4;
            Slot at;
            int local = 0;
            bool ok = true, issued = false;
            for (long long j = pair0; j < p.jobs && ok; j += pairs, ++local) {
                const int tile = (int)(j / p.NT) * kPairRows, buf = local & 1;
                if (local >= 2 && !wait_or_abort(sm.acc_empty + 8 * buf, ((local >> 1) - 1) & 1, sm.abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t dcol = tmem + (uint32_t)(buf * p.BN);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!wait_or_abort(sm.full + 8 * at.s, at.pass & 1, sm.abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = a0 + at.s * sstep, bd = b0 + at.s * sstep;
                    mma_pair(dcol, ad, bd, idesc, kb != kb0);
                    mma_pair(dcol, ad + 2, bd + 2, idesc, 1u);
                    mma_pair(dcol, ad + 4, bd + 4, idesc, 1u);
                    mma_pair(dcol, ad + 6, bd + 6, idesc, 1u);
                    issued = true;
                    commit_pair(sm.empty + 8 * at.s, leader);
                    at.next(p.stages);
                }
                for (RequestsOf w(req, tile, tile + kPairRows); adapters && ok && w.valid(); w.next()) {
                    if (w.hi <= w.lo || req.adapter(w.r) < 0) continue;
                    const int r0 = w.lo - tile, r1 = w.hi - tile;  // this request's rows of the tile
                    uint32_t off[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) off[i] = ~lane_bits(r0 - 32 * i, r1 - 32 * i);
                    for (int st = 0; st < RB * 2 / held; ++st) {  // a block of rank: both values of t, or one after the other
                        if (!wait_or_abort(sm.full + 8 * at.s, at.pass & 1, sm.abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t ad = a1 + at.s * sstep, bd = b1 + at.s * sstep;
                        const int steps = min(4, (p.rank - st * held / 2 * kBK + 15) / 16);
                        for (int v = 0; v < held; ++v)
                            for (int i = 0; i < steps; ++i)
                                mma_pair_rows(dcol, ad + (uint32_t)(v * kBM * p.aw >> 4) + 2 * i, bd + 2 * i, idesc, off);
                        commit_pair(sm.empty + 8 * at.s, leader);
                        at.next(p.stages);
                    }
                }
                if (!ok) break;
                commit_pair(sm.acc_full + 8 * buf, leader);
            }
            if (!ok) raise_abort(sm.abort_flag, p.err);
            if (issued) {
                // every product has finished before tensor memory is freed
                commit_pair(sm.drain, leader);
                mbar_wait_bounded(sm.drain, 0, kTcWaitNs);
            }
        }
        __syncwarp();
    } else {
        // ---- epilogue: this CTA's rows, warp w the tensor-memory lanes 32 * (w % 4) .. +31, two warps taking the
        // 64-column chunks in turn.  A chunk goes through shared memory and out by TMA in whole lines (16-byte
        // stores by lanes that each own a row touch 32 lines an instruction); rows of no request are not to be
        // written, so a warp that holds some stores by lanes instead.
        const int quad = warp & 3, half = (warp - 2) >> 2;
        const T *bias = static_cast<const T *>(p.bias);
        const int covered0 = req.at(0), covered1 = req.at(p.requests);
        const uint32_t acc_empty0 = in_cta(sm.acc_empty, leader);
        unsigned char *own = sm.ring + p.stages * sbytes + (warp - 2) * kOutBytes;  // box of 4 KB
        const uint32_t stage = smem_u32(own);
        float *bias_s = reinterpret_cast<float *>(sm.ring + p.stages * sbytes + 8 * kOutBytes) + (warp - 2) * kBK;
        int local = 0;
        if (p.shift) asm volatile("griddepcontrol.wait;" ::: "memory");  // SHRINK's exponents are there
        for (long long j = pair0; j < p.jobs; j += pairs, ++local) {
            const int row0 = (int)(j / p.NT) * kPairRows + rank * kBM + quad * 32, row = row0 + lane;
            const int n0 = (int)(j % p.NT) * p.BN, ncols = min(p.BN, p.cout - n0), buf = local & 1;
            // the map ends at the last row: rows past it are not written either way
            const bool boxes = row0 >= covered0 && min(row0 + 32, p.rows) <= covered1;
            const bool write = row >= covered0 && row < covered1;
            const int far = shifted_row(row, write);
            const bool shifted = kShifted && __any_sync(0xffffffffu, far >= 0);
            bool ready = false;
            if (p.splits > 1) {
                if (!wait_or_abort(sm.acc_full, 0, sm.abort_flag)) {
                    raise_abort(sm.abort_flag, p.err);
                    break;
                }
                tc_fence_after();
                // the products have read the ring
                dump_accumulator(tmem + ((uint32_t)(32 * quad) << 16), reinterpret_cast<float *>(sm.ring) + quad * 32 + lane,
                                 p.BN, 16 * half, 32);
                break;
            }
            for (int c = half * kBK; c < ncols; c += 2 * kBK) {  // warp-uniform
                __syncwarp();
                for (int i = lane; i < kBK; i += 32)
                    bias_s[i] = bias && c + i < ncols ? to_f32(bias[n0 + c + i]) : 0.0f;
                // the box that was staged here before has been read
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
                if (!ready) {
                    if (!wait_or_abort(sm.acc_full + 8 * buf, (local >> 1) & 1, sm.abort_flag)) break;
                    tc_fence_after();
                    ready = true;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v[32];
                    tmem_ld32(tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(buf * p.BN + c + 32 * h), v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 b = reinterpret_cast<const float4 *>(bias_s)[8 * h + i];
                        v[4 * i] += b.x;
                        v[4 * i + 1] += b.y;
                        v[4 * i + 2] += b.z;
                        v[4 * i + 3] += b.w;
                    }
                    if (shifted) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (far >= 0 && c + 32 * h + i < ncols) v[i] += missing(row, far, n0 + c + 32 * h + i);
                        __syncwarp();
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 q = pack16<T>(v + 8 * i);
                        const int col = c + 32 * h + 8 * i;
                        if (boxes)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                             stage + (uint32_t)(lane * 128 + (((4 * h + i) ^ (lane & 7)) << 4))),
                                         "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w)
                                         : "memory");
                        else if (write && col < ncols)  // cout is a multiple of 8
                            *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + (long long)row * p.cout + n0 + col) = q;
                    }
                }
                if (boxes) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) tma_store_2d(&ymap, stage, n0 + c, row0);
                }
            }
            // a warp without a chunk still takes part in every accumulator's turn
            if (!ready && !wait_or_abort(sm.acc_full + 8 * buf, (local >> 1) & 1, sm.abort_flag)) {
                raise_abort(sm.abort_flag, p.err);
                break;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_remote(acc_empty0 + 8 * buf);
        }
        // the boxes have left shared memory; the end of the kernel completes their writes
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
    }
    if (p.splits > 1) {
        __syncwarp();
        cluster_sync();
        if (warp >= 2 && pair0 < p.jobs) {
            // this split's share of the columns, 8 at a time; the row is the lane's
            const int quad = warp & 3, half = (warp - 2) >> 2;
            const int row = (int)(pair0 / p.NT) * kPairRows + rank * kBM + quad * 32 + lane;
            const int n0 = (int)(pair0 % p.NT) * p.BN, ncols = min(p.BN, p.cout - n0);
            const bool write = row >= req.at(0) && row < req.at(p.requests);
            const int far = shifted_row(row, write);
            const uint32_t addr = smem_u32(sm.ring) + (uint32_t)(quad * 32 + lane) * 4;
            for (int c = 8 * (split * 2 + half); c < ncols; c += 16 * p.splits) {
                float v[8], b[8] = {};
                if (p.bias) unpack16<T>(ld_nc16(static_cast<const T *>(p.bias) + n0 + c), b);
                add_splits(addr, c, p.splits, rank, 2, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += b[i];
                if (far >= 0) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] += missing(row, far, n0 + c + i);
                }
                if (write)
                    *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + (long long)row * p.cout + n0 + c) = pack16<T>(v);
            }
        }
        __syncwarp();
    }
    // a pair that had no t to wait for still ends after SHRINK: the next user of the workspace is ordered behind
    // this kernel
    asm volatile("griddepcontrol.wait;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA frees or leaves what the other still uses
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols)
                     : "memory");
    }
}

template <typename T> CUtensorMapDataType data_type() {
    return std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}
CUtensorMapSwizzle swizzle_of(int width) {
    return width == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : width == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
}

// Boxes of `box` rows and `width` bytes over a [rows, cols] matrix of T, in the swizzle of that width.
template <typename T>
bool encode(CUtensorMap *m, const void *base, long long cols, long long rows, int box, int width = 128) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t str[1] = {(cuuint64_t)cols * 2};
    const cuuint32_t bx[2] = {(cuuint32_t)(width / 2), (cuuint32_t)box}, es[2] = {1, 1};
    return encode_fn()(m, data_type<T>(), 2, const_cast<void *>(base), dims, str, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       swizzle_of(width), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// t of a pass: boxes of 128 rows of as many of its two values as a stage holds.
template <typename T> bool encode_t(CUtensorMap *m, const void *base, int rank, int rows, int width) {
    const cuuint64_t dims[3] = {(cuuint64_t)rank, (cuuint64_t)rows, 2};
    const cuuint64_t str[2] = {(cuuint64_t)rank * 2, (cuuint64_t)rows * rank * 2};
    const cuuint32_t bx[3] = {(cuuint32_t)(width / 2), kBM, width < 128 ? 2u : 1u}, es[3] = {1, 1, 1};
    return encode_fn()(m, data_type<T>(), 3, const_cast<void *>(base), dims, str, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       swizzle_of(width), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int tmem_columns(int bn) {
    int cols = 32;
    while (cols < 2 * bn) cols <<= 1;
    return cols;
}

// Stages of `sbytes` that fit and that a CTA's `use` blocks can fill (a short ring leaves EXPAND room beside SHRINK's
// last CTAs), and the shared memory they take with `extra`; the accumulator of a split, `sums` bytes, takes the ring's
// place.
size_t plan_smem(LargeParams &p, size_t sbytes, size_t sums, size_t extra, size_t limit, long long use) {
    const size_t other = extra + 1024 + (2 * kMaxStages + 5) * 8 + 8 +
                         (p.requests <= kReqCache ? (size_t)(2 * p.requests + 1) * 4 : 0);
    p.stages = use < 2 ? 2 : use < kMaxStages ? (int)use : kMaxStages;
    while (p.stages > 2 && other + p.stages * sbytes > limit) --p.stages;
    if (p.splits > 1)
        while (p.stages * sbytes < sums && p.stages < kMaxStages) ++p.stages;
    const size_t need = other + p.stages * sbytes, share = tensor_memory_share(limit, p.tmem_cols);
    const size_t least = p.splits > 1 && share < limit / 4 ? limit / 4 : share;  // (a pair's staged output takes more)
    return need > least ? need : least;
}

// Bytes of t for one row: two values of the storage type for each rank, and in fp16 the exponents.
size_t t_bytes(const AdapterArgs &a) { return (size_t)a.rank * 4 + (a.dtype == DType::F16 ? kShiftBytes : 0); }

// One pass over rows row0 .. row0 + a.rows - 1 of the request table; x and out of `a` start there.
template <typename T> cudaError_t launch_pass(const AdapterArgs &a, int row0, cudaStream_t stream) {
    const DeviceInfo *dev = device_info();
    if (!encode_fn() || !dev) return cudaErrorNotSupported;
    LargeParams p;
    p.row0 = row0;
    p.rows = (int)a.rows;
    p.cin = a.cin; p.cout = a.cout; p.rank = a.rank; p.adapters = a.adapters; p.requests = a.requests;
    p.start = a.start; p.which = a.which; p.scale = a.scale; p.bias = a.bias;
    p.t = a.workspace;
    p.shift = a.dtype == DType::F16 && a.adapters > 0
                  ? static_cast<unsigned char *>(a.workspace) + (size_t)a.rows * a.rank * 4
                  : nullptr;
    p.b = a.b;
    p.out = a.out;
    p.err = dev->err;

    // Tile width and splits of the contraction by their cost in clocks of an SM, as measured: 2.6 for each 64-wide
    // row that it fetches (128 of x, half a tile of W, a block of the contraction), 12 for each column of the
    // epilogue, 1500 for a round of tiles, 10000 for the exchange between splits.  Clusters that split have one tile.
    const long long mt = (a.rows + kPairRows - 1) / kPairRows, pairs = dev->sms / 2;
    const int blocks = (a.cin + kBK - 1) / kBK;
    int bn = 0, splits = 1;
    double best = 0.0;
    for (int c = 256; c >= 64; c /= 2)
        for (int s = 1; s <= 4 && s <= blocks; s *= 2) {
            const long long tiles = mt * ((a.cout + c - 1) / c);
            if (s > 1 && tiles * s > kClusterPairs) break;
            const double rounds = s > 1 ? 1.0 : (double)((tiles + pairs - 1) / pairs);
            const double cost = rounds * (1500.0 + 2.6 * ((blocks + s - 1) / s) * (128 + c / 2) + 12.0 * c) + (s > 1 ? 10000.0 : 0.0);
            if (!bn || cost < best) {
                bn = c;
                splits = s;
                best = cost;
            }
        }
    const int rank16 = (a.rank + 15) / 16 * 16;
    // low ranks in rows of their own width: boxes of 128 bytes that are mostly fill cost as much as full ones
    // (256 -> 4096, 80 rows: 23 us at rank 16 against 16 at rank 64)
    p.aw = a.rank <= 16 ? 32 : a.rank <= 32 ? 64 : 128;
    CUtensorMap xm, am, wm, tm, bm, ym;
    if (!encode<T>(&xm, a.x, a.cin, a.rows, kBM) || !encode<T>(&wm, a.weight, a.cin, a.cout, bn / 2) ||
        !encode<T>(&ym, a.out, a.cout, a.rows, 32))
        return cudaErrorInvalidValue;
    am = tm = bm = wm;  // never read without adapters
    if (a.adapters > 0 && (!encode<T>(&am, a.a, a.cin, (long long)a.adapters * a.rank, rank16) ||
                           !encode_t<T>(&tm, a.workspace, a.rank, (int)a.rows, p.aw) ||
                           !encode<T>(&bm, a.b, a.rank, (long long)a.adapters * a.cout, bn / 2, p.aw)))
        return cudaErrorInvalidValue;

    static std::atomic<bool> shrink_ok[kMaxDev], expand_ok[kMaxDev];
    cudaError_t e = allow_smem(adapters_shrink_kernel<T>, dev->smem_optin, shrink_ok);
    if (e == cudaSuccess) e = allow_smem(adapters_expand_kernel<T>, dev->smem_optin, expand_ok);
    if (e != cudaSuccess) return e;
    p.BN = rank16;
    p.NT = 1;
    p.jobs = (a.rows + kBM - 1) / kBM + a.requests;
    p.splits = 1;
    // the exchange costs 2 us, what 8 blocks take: halve runs of 16 blocks and more, where EXPAND's CTAs still find
    // SMs beside SHRINK's (128 rows 4096 -> 4096, rank 64: 33 us beside it, 42 behind it)
    const long long expand_ctas = 2 * splits * mt * ((a.cout + bn - 1) / bn);
    while (p.splits < 8 && 2 * p.splits * p.jobs + expand_ctas <= dev->sms && blocks >= 16 * p.splits) p.splits *= 2;
    p.tmem_cols = tmem_columns(p.BN);
    size_t smem = plan_smem(p, kABytes + p.BN * kBK * 2, (size_t)p.BN * kBM * 4, 0, (size_t)dev->smem_optin,
                            (blocks + p.splits - 1) / p.splits * ((p.jobs + dev->sms - 1) / dev->sms));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.stream = stream;
    cfg.gridDim = dim3((unsigned)(p.splits > 1 ? p.jobs * p.splits : p.jobs < dev->sms ? p.jobs : dev->sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, adapters_shrink_kernel<T>, xm, am, p);
    if (e != cudaSuccess) return e;

    p.BN = bn;
    p.NT = (a.cout + bn - 1) / bn;
    p.jobs = mt * p.NT;
    p.splits = splits;
    p.tmem_cols = tmem_columns(p.BN);
    smem = plan_smem(p, kABytes + p.BN / 2 * kBK * 2, (size_t)p.BN * kBM * 4, kOutStage, (size_t)dev->smem_optin,
                     ((blocks + splits - 1) / splits + 2) * ((p.jobs + pairs - 1) / pairs));
    attr[0].val.clusterDim.x = (unsigned)(2 * splits);
    cfg.gridDim = dim3((unsigned)(2 * splits * (p.jobs < pairs ? p.jobs : pairs)));
    cfg.blockDim = dim3(kExpandThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, adapters_expand_kernel<T>, xm, wm, tm, bm, ym, p);
}

}  // namespace

size_t adapters_large_workspace(const AdapterArgs &a) { return (size_t)a.rows * a.rank * 2; }

cudaError_t launch_adapters_large(const AdapterArgs &a, cudaStream_t stream) {
    if (a.dtype != DType::F16 && a.dtype != DType::BF16) return cudaErrorInvalidValue;
    // as many rows in a pass as the workspace holds t of, in whole tiles where that is more than one
    const int64_t fit = (int64_t)(a.workspace_bytes / t_bytes(a));
    const int64_t step = fit >= a.rows ? a.rows : fit >= kPairRows ? fit / kPairRows * kPairRows : fit;
    if (step < 1) return cudaErrorInvalidValue;
    AdapterArgs g = a;
    for (int64_t row0 = 0; row0 < a.rows; row0 += step) {
        g.rows = a.rows - row0 < step ? a.rows - row0 : step;
        g.x = static_cast<const char *>(a.x) + row0 * a.cin * 2;
        g.out = static_cast<char *>(a.out) + row0 * a.cout * 2;
        const cudaError_t e = a.dtype == DType::F16 ? launch_pass<__half>(g, (int)row0, stream)
                                                    : launch_pass<__nv_bfloat16>(g, (int)row0, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// The route by its time in microseconds, as measured (one B200; cin and cout of 256 to 4096, ranks 16 to 128).  The
// row-wise route (dcn_proj_adapters_rows.cu): 6.5, the weight at 5 TB/s, 0.02 a row for the partial sums, and 2.4
// million products a microsecond for t and the adapter term, which do not use the tensor cores.  The tiles of this
// file: 12, 0.36 for each block of the contraction and round of tiles, and for each further request, whose blocks
// of t and B follow one another, 0.4 and 0.55 for each stage that they take (1024 -> 1024, rank 64, 256 rows: of one
// request 22.9 and 14.8, of 16 22.9 and 35.8, of 256 24.3 and 395).  Up to 64 rows it is always the first.
static bool few_rows(const AdapterArgs &a) {
    if (a.rows <= 64) return true;
    if (a.rows > kMaxSmallRows) return false;
    const double rows = 6.5 + 2.0 * a.cin * a.cout / 5.0e6 + 0.02 * (double)a.rows +
                        (double)a.rows * a.rank * ((double)a.cin + a.cout) / 2.4e6;
    const int blocks = (a.cin + kBK - 1) / kBK, tiles = (a.cout + 63) / 64, rounds = (tiles + 73) / 74;
    const int further = (int)(a.requests < a.rows ? a.requests : a.rows) - 1;  // as many at most as own rows
    const int stages = a.rank <= 32 ? 1 : 2 * ((a.rank + kBK - 1) / kBK);
    return rows <= 12.0 + 0.36 * blocks * rounds + further * (0.4 + 0.55 * stages);
}

size_t proj_adapters_workspace(const AdapterArgs &a) {
    return few_rows(a) ? adapters_small_workspace(a) : adapters_large_workspace(a);
}

size_t proj_adapters_workspace_full(const AdapterArgs &a) {
    return few_rows(a) ? adapters_small_workspace(a) : (size_t)a.rows * t_bytes(a);
}

cudaError_t launch_proj_adapters(const AdapterArgs &a, cudaStream_t stream) {
    return few_rows(a) ? launch_adapters_small(a, stream) : launch_adapters_large(a, stream);
}

}  // namespace dcnb
