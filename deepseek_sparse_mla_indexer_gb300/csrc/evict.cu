// Eviction from a paged cache by accumulated attention weight:
//   nsa_evict_select   which positions of each request stay
//   nsa_evict_compact  the kept rows of every paged array moved to the front
//
// The totals are what nsa_mla_key_weights sums.  A request of length L over
// its budget keeps its first `sinks` positions, its last `recent` ones, and of
// those between the budget - sinks - recent with the largest totals (equal
// totals prefer the lower position, -0 equals +0, NaN ranks lowest, as the
// top-k ranks scores).
#include "nsa_internal.cuh"
#include "sm100.cuh"

namespace nsa {
namespace {

using namespace sm100;

// ------------------------------------------------------------------ select
//
// One thread-block cluster per request; its CTAs own equal slices of the
// positions.  The threshold key of the middle range is found by a radix
// selection over 11 + 11 + 10 bits of the order-preserving key: each CTA counts
// its slice's digits in shared memory, each sums one part of the bins over the
// cluster (distributed shared memory), and the CTA whose part holds the
// threshold tells the others the digit and how many keys remain to be taken
// from it.  Then every CTA writes its kept positions behind those of the CTAs
// before it: positions above the threshold, and of those equal to it the lowest
// ones.  Keys are read from HBM once (they stay in shared memory where a slice
// fits), so a long row costs one pass plus about ten cluster barriers; whole
// numbers throughout, so the result does not depend on scheduling.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelMaxCluster = 8;         // the portable limit
constexpr int kSelCache = 48 * 1024;      // keys of a slice kept in shared memory
constexpr int kSelSlice = 4096;           // positions per CTA that the cluster size aims for
constexpr int kSelPer = 2048 / kSelThreads;  // consecutive bins a thread sums

struct SelShared {
    uint32_t hist[2048];
    uint32_t seg[kSelMaxCluster];          // bins summed over the cluster, per part
    uint32_t digit, need;                  // written by the part that holds the threshold
    uint32_t warp_sure[kSelWarps], warp_eq[kSelWarps];
    uint32_t cta_sure, cta_eq;             // this CTA's counts, read by the others
    uint32_t scan[kSelWarps];
};

__device__ __forceinline__ uint32_t dsmem_ld_u32(const uint32_t *local, uint32_t rank)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(dsmem_addr(local, rank)) : "memory");
    return v;
}
__device__ __forceinline__ void dsmem_st_u32(uint32_t *local, uint32_t rank, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dsmem_addr(local, rank)), "r"(v) : "memory");
}

// Adds 1 to hist[bin] for every lane with `on`; a warp whose lanes all name one
// bin (rows of equal totals) adds once.
__device__ __forceinline__ void count_digit(uint32_t *hist, uint32_t bin, bool on, int lane)
{
    int all;
    __match_all_sync(0xffffffffu, on ? bin : 0xffffffffu, &all);
    if (all) {
        if (on && lane == 0) atomicAdd(hist + bin, 32u);
    } else if (on) {
        atomicAdd(hist + bin, 1u);
    }
}

__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const float *total, int64_t total_ld, const int32_t *lens, int max_len, int sinks, int recent,
                    int budget, int slice, int cached, int32_t *keep, int64_t keep_ld, int32_t *new_len, int32_t *status)
{
    extern __shared__ uint32_t key_s[];  // [slice] order keys when `cached`
    __shared__ SelShared sm;
    const int nc = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
    const int b = blockIdx.x / nc;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int32_t *out = keep + (int64_t)b * keep_ld;
    int L = lens[b];
    if (L < 0 || L > max_len) {
        if (rank == 0 && tid == 0) set_status(status, NSA_ERR_BOUNDS);
        L = 0;
    }
    if (L <= budget) {  // nothing to evict (uniform over the cluster: no barrier is skipped)
        for (int i = rank * kSelThreads + tid; i < budget; i += nc * kSelThreads) out[i] = i < L ? i : -1;
        if (rank == 0 && tid == 0) new_len[b] = L;
        return;
    }
    const float *row = total + (int64_t)b * total_ld;
    const int mid0 = sinks, mid1 = L - recent;  // the middle range; sinks + recent <= budget < L
    const int p0 = min(L, rank * slice), p1 = min(L, p0 + slice);
    const int m0 = min(p1, max(p0, mid0)), m1 = max(m0, min(p1, mid1));  // its part of this slice
    auto key_at = [&](int i) -> uint32_t { return cached ? key_s[i - p0] : order_key(__ldg(row + i)); };

    uint32_t need = (uint32_t)(budget - sinks - recent), prefix = 0;
    const bool any = need > 0;  // else nothing between the ends is kept
    if (any) {
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const int bins = pass == 2 ? 1024 : 2048;
            for (int i = tid; i < bins; i += kSelThreads) sm.hist[i] = 0;
            __syncthreads();
            // whole warps step together (count_digit is a warp operation)
            for (int i0 = m0 + warp * 32; i0 < m1; i0 += kSelThreads * 4) {
                uint32_t k[4];
                bool on[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int i = i0 + u * kSelThreads + lane;
                    on[u] = i < m1;
                    k[u] = on[u] ? (pass == 0 ? order_key(__ldg(row + i)) : key_at(i)) : 0u;
                    if (pass == 0 && cached && on[u]) key_s[i - p0] = k[u];
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const bool in = on[u] && (pass == 0 || (k[u] >> (shift + (pass == 1 ? 11 : 10))) == prefix);
                    count_digit(sm.hist, (k[u] >> shift) & (uint32_t)(bins - 1), in, lane);
                }
            }
            cluster_sync_all();  // every CTA's counts are complete
            // part `rank` of the bins, summed over the cluster, kSelPer consecutive bins a thread
            const int per = bins / nc;
            uint32_t tot[kSelPer];
            uint32_t sum = 0;
#pragma unroll
            for (int u = 0; u < kSelPer; ++u) {
                tot[u] = 0;
                const int x = tid * kSelPer + u;
                if (x < per)
                    for (int q = 0; q < nc; ++q) tot[u] += dsmem_ld_u32(sm.hist + rank * per + x, (uint32_t)q);
                sum += tot[u];
            }
            // suffix sums over the threads (higher bins first)
            uint32_t suf = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_down_sync(0xffffffffu, suf, o);
                if (lane + o < 32) suf += v;
            }
            if (lane == 0) sm.scan[warp] = suf;
            __syncthreads();
            uint32_t above = suf - sum;
            for (int w = warp + 1; w < kSelWarps; ++w) above += sm.scan[w];
            if (tid < nc) {
                uint32_t all = 0;
                for (int w = 0; w < kSelWarps; ++w) all += sm.scan[w];
                dsmem_st_u32(sm.seg + rank, (uint32_t)tid, all);
            }
            cluster_sync_all();  // every part's sum is known everywhere
            for (int q = rank + 1; q < nc; ++q) above += sm.seg[q];
            // the bin where the count from the top reaches `need`: exactly one thread of the cluster has it
#pragma unroll
            for (int u = kSelPer - 1; u >= 0; --u) {
                if (above < need && above + tot[u] >= need) {
                    const uint32_t d = (uint32_t)(rank * per + tid * kSelPer + u);
                    for (int q = 0; q < nc; ++q) {
                        dsmem_st_u32(&sm.digit, (uint32_t)q, d);
                        dsmem_st_u32(&sm.need, (uint32_t)q, need - above);
                    }
                }
                above += tot[u];
            }
            cluster_sync_all();  // digit and need have arrived; hist may be cleared
            prefix = (prefix << (pass == 2 ? 10 : 11)) | sm.digit;
            need = sm.need;
        }
    }
    const uint32_t threshold = prefix;
    // count, per warp over its contiguous part, the positions surely kept and those equal to the threshold
    const int len = p1 - p0, per_warp = ((len + kSelWarps * 32 - 1) / (kSelWarps * 32)) * 32;
    const int w0 = min(p1, p0 + warp * per_warp), w1 = min(p1, w0 + per_warp);
    auto classify = [&](int i, bool &sure, bool &eq) {
        const bool in = i < w1, mid = in && i >= mid0 && i < mid1;
        const uint32_t k = mid && any ? key_at(i) : 0u;
        sure = in && (!mid || (any && k > threshold));
        eq = mid && any && k == threshold;
    };
    uint32_t n_sure = 0, n_eq = 0;
    for (int i0 = w0; i0 < w1; i0 += 32) {
        bool sure, eq;
        classify(i0 + lane, sure, eq);
        n_sure += __popc(__ballot_sync(0xffffffffu, sure));
        n_eq += __popc(__ballot_sync(0xffffffffu, eq));
    }
    if (lane == 0) {
        sm.warp_sure[warp] = n_sure;
        sm.warp_eq[warp] = n_eq;
    }
    __syncthreads();
    uint32_t eq_before = 0, sure_before = 0, cta_eq = 0, cta_sure = 0;
    for (int w = 0; w < kSelWarps; ++w) {
        if (w < warp) {
            eq_before += sm.warp_eq[w];
            sure_before += sm.warp_sure[w];
        }
        cta_eq += sm.warp_eq[w];
        cta_sure += sm.warp_sure[w];
    }
    if (tid == 0) {
        sm.cta_eq = cta_eq;
        sm.cta_sure = cta_sure;
    }
    cluster_sync_all();
    for (int q = 0; q < rank; ++q) {
        eq_before += dsmem_ld_u32(&sm.cta_eq, (uint32_t)q);
        sure_before += dsmem_ld_u32(&sm.cta_sure, (uint32_t)q);
    }
    // a position's place: the sure ones before it plus the equal ones taken before it
    for (int i0 = w0; i0 < w1; i0 += 32) {
        bool sure, eq;
        classify(i0 + lane, sure, eq);
        const uint32_t below = (1u << lane) - 1u;
        const uint32_t bs = __ballot_sync(0xffffffffu, sure), be = __ballot_sync(0xffffffffu, eq);
        const uint32_t e = eq_before + __popc(be & below);
        const uint32_t at = sure_before + __popc(bs & below) + min(e, need);
        if (sure || (eq && e < need)) out[at] = i0 + lane;
        eq_before += __popc(be);
        sure_before += __popc(bs);
    }
    if (rank == 0 && tid == 0) new_len[b] = budget;
    cluster_sync_all();  // a peer may still read this CTA's counts
}

// ------------------------------------------------------------------ compact
//
// Position i of a request's front takes the row of position keep[i], in place.
// keep ascends, so keep[i] >= i: rows only move towards the front, and a row
// may be overwritten as soon as it has been read.  The positions are cut into
// chunks of T; a CTA stages its chunk's source rows in shared memory, announces
// that it has read them, waits until every chunk that reads rows from its own
// destination range has announced the same, and writes.  Those are chunks with
// lower numbers (keep[j] >= j), at most two besides itself (each spans at least
// T source positions), and chunks are handed out in ascending order, so the
// waits end: the lowest unfinished chunk never waits.  Bound by HBM: every row
// that moves is read and written once; rows that stay are not touched.
constexpr int kMaxArrays = 8;
constexpr int kCpThreads = 256;
constexpr int kCpMinT = 8, kCpMaxT = 128;
constexpr int kCpStage = 56 * 1024;      // bytes staged per CTA: four CTAs per SM
constexpr int kCpMaxRow = 24 * 1024;     // bytes of one position over all arrays
constexpr long long kCpWait = 2000000000LL;  // ~1 s of SM clocks

struct CompactParams {
    uint8_t *array[kMaxArrays];
    int row_bytes[kMaxArrays];
    int unit[kMaxArrays];       // bytes per copy step: 16, 4 or 1
    int offset[kMaxArrays];     // of the array's rows within the stage
    int n_arrays;
    const int32_t *keep;
    int64_t keep_ld;
    const int32_t *new_len, *old_len;
    const int32_t *page_table;
    int64_t pt_ld;
    int page_size, max_len, budget;
    int64_t num_pages;
    float *total;
    int64_t total_ld;
    int T, chunks, B;
    int32_t *read_done;  // [B][chunks], zero at the start
    int32_t *ticket;     // zero at the start
    int32_t *status;
};

__device__ __forceinline__ int ld_acquire(const int32_t *p)
{
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_release(int32_t *p, int v)
{
    asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// The number of entries of the ascending keep[0 .. n) below `v`, by the whole CTA.
__device__ __forceinline__ int block_lower_bound(const int32_t *keep, int n, int v)
{
    int lo = 0, len = n;  // the answer lies in [lo, lo + len]
    while (len > 0) {
        const int step = (len + kCpThreads - 1) / kCpThreads;
        const int i = (int)threadIdx.x * step;
        const int c = __syncthreads_count(i < len && keep[lo + i] < v);
        if (c == 0) return lo;
        if (step == 1) return lo + c;
        lo += (c - 1) * step + 1;  // entry (c - 1) * step is below v
        len = min(step - 1, len - (c - 1) * step - 1);
    }
    return lo;
}

template <int UNIT> struct CopyUnit;
template <> struct CopyUnit<16> { using type = uint4; };
template <> struct CopyUnit<4> { using type = uint32_t; };
template <> struct CopyUnit<1> { using type = uint8_t; };

// Rows of one array between the cache and the stage.
template <int UNIT, bool READ>
__device__ __forceinline__ void move_rows(uint8_t *array, int row_bytes, uint8_t *stage, const int64_t *slot, int T)
{
    using U = typename CopyUnit<UNIT>::type;
    const int per = row_bytes / UNIT;
    for (int e = threadIdx.x; e < T * per; e += kCpThreads) {
        const int i = e / per, c = e - i * per;
        if (slot[i] < 0) continue;
        U *g = reinterpret_cast<U *>(array + slot[i] * row_bytes) + c;
        U *s = reinterpret_cast<U *>(stage + (int64_t)i * row_bytes) + c;
        if constexpr (READ && UNIT == 16)
            cp_async16(s, g);
        else if constexpr (READ)
            *s = __ldcg(g);
        else
            *g = *s;
    }
}

template <bool READ>
__device__ __forceinline__ void move_all(const CompactParams &p, uint8_t *stage, const int64_t *slot)
{
    for (int a = 0; a < p.n_arrays; ++a) {
        if (p.unit[a] == 16)
            move_rows<16, READ>(p.array[a], p.row_bytes[a], stage + p.offset[a], slot, p.T);
        else if (p.unit[a] == 4)
            move_rows<4, READ>(p.array[a], p.row_bytes[a], stage + p.offset[a], slot, p.T);
        else
            move_rows<1, READ>(p.array[a], p.row_bytes[a], stage + p.offset[a], slot, p.T);
    }
}

__global__ void __launch_bounds__(kCpThreads) evict_compact_kernel(CompactParams p)
{
    extern __shared__ __align__(16) uint8_t stage[];
    __shared__ int64_t src[kCpMaxT], dst[kCpMaxT];  // slots of the chunk's rows; -1: does not move
    __shared__ int s_ticket, s_timeout;
    const int tid = threadIdx.x;
    const int n_tickets = p.B * p.chunks;
    if (tid == 0) s_timeout = 0;
    for (;;) {
        __syncthreads();  // the stage and the slot lists are free
        if (tid == 0) s_ticket = atomicAdd(p.ticket, 1);
        __syncthreads();
        const int ticket = s_ticket;
        if (ticket >= n_tickets) return;
        // tickets go round the requests first: a chunk's predecessors are then well ahead of it
        const int c = ticket / p.B, b = ticket - c * p.B;
        const int old = p.old_len[b], n = p.new_len[b];
        const bool bad = old < 0 || old > p.max_len || n < 0 || n > old || n > p.budget;
        if (bad && tid == 0 && c == 0) set_status(p.status, NSA_ERR_BOUNDS);
        const int lo = c * p.T, hi = min(old, lo + p.T);
        if (bad || n == old || lo >= (p.total ? old : n)) continue;  // uniform over the CTA
        const int32_t *keep = p.keep + (int64_t)b * p.keep_ld;
        const int32_t *pt = p.page_table + (int64_t)b * p.pt_ld;
        float *total = p.total ? p.total + (int64_t)b * p.total_ld : nullptr;
        float t = 0.f;  // the total that moves to (or, past the kept rows, clears) position lo + tid
        if (tid < p.T) {
            const int i = lo + tid;
            int64_t s = -1, d = -1;
            if (i < n) {
                const int k = keep[i];
                if (k < i || k >= old || (i > 0 && keep[i - 1] >= k)) {
                    set_status(p.status, NSA_ERR_BOUNDS);  // not an ascending list of positions
                    if (total) t = __ldcg(total + i);
                } else {
                    if (total) t = __ldcg(total + k);
                    if (k != i && p.n_arrays > 0) {
                        const int32_t ps = pt[k / p.page_size], pd = pt[i / p.page_size];
                        if (ps < 0 || ps >= p.num_pages || pd < 0 || pd >= p.num_pages) {
                            set_status(p.status, NSA_ERR_BOUNDS);
                        } else {
                            s = (int64_t)ps * p.page_size + k % p.page_size;
                            d = (int64_t)pd * p.page_size + i % p.page_size;
                        }
                    }
                }
            }
            src[tid] = s;
            dst[tid] = d;
        }
        __syncthreads();
        move_all<true>(p, stage, src);
        cp_async_commit();
        // while the rows are under way: rows j0 .. j1-1 are those read from this chunk's range
        const int j0 = block_lower_bound(keep, n, lo), j1 = block_lower_bound(keep, n, hi);
        cp_async_wait_all();
        __syncthreads();  // every thread's reads (rows and totals) have arrived
        int32_t *done = p.read_done + (int64_t)b * p.chunks;
        if (tid == 0) {
            __threadfence();
            st_release(done + c, 1);
            if (j1 > j0) {
                for (int x = j0 / p.T; x <= (j1 - 1) / p.T && x < c; ++x) {
                    const long long t0 = clock64();
                    while (!ld_acquire(done + x)) {
                        if (clock64() - t0 > kCpWait) {
                            set_status(p.status, NSA_ERR_TIMEOUT);
                            s_timeout = 1;
                            break;
                        }
                        __nanosleep(64);
                    }
                }
            }
        }
        __syncthreads();
        if (s_timeout) return;  // rows that another chunk may not have read are left as they are
        move_all<false>(p, stage, dst);
        if (total && tid < p.T && lo + tid < hi) total[lo + tid] = t;
    }
}

}  // namespace
}  // namespace nsa

extern "C" nsa_status nsa_evict_select(const float *total_dev, int64_t total_ld, const int32_t *len_dev, int B,
                                       int max_len, int sinks, int recent, int budget, int32_t *keep_dev,
                                       int64_t keep_ld, int32_t *new_len_dev, int32_t *status_dev, nsa_stream_t stream)
{
    using namespace nsa;
    if (B < 0 || max_len < 0 || sinks < 0 || recent < 0 || budget < 1 || keep_ld < budget || total_ld < max_len)
        return NSA_ERR_INVALID_ARG;
    if ((int64_t)sinks + recent > budget) return NSA_ERR_INVALID_ARG;
    if (max_len > (1 << 30)) return NSA_ERR_UNSUPPORTED;
    if (B == 0) return NSA_OK;
    if (!len_dev || !keep_dev || !new_len_dev || (max_len > 0 && !total_dev)) return NSA_ERR_INVALID_ARG;
    if (((uintptr_t)total_dev | (uintptr_t)len_dev | (uintptr_t)keep_dev | (uintptr_t)new_len_dev |
         (uintptr_t)status_dev) & 3)
        return NSA_ERR_INVALID_ARG;
    int nc = 1;
    while (nc < kSelMaxCluster && (int64_t)nc * kSelSlice < max_len) nc *= 2;
    if ((int64_t)B * nc > 0x7fffffffLL) return NSA_ERR_UNSUPPORTED;
    const int slice = max_len > 0 ? (int)ceil_div(max_len, nc) : 1;
    const int cached = slice <= kSelCache ? 1 : 0;
    NSA_CUDA_TRY(cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelCache * 4));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * nc));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = cached ? (size_t)slice * 4 : 0;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)nc;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    NSA_CUDA_TRY(cudaLaunchKernelEx(&cfg, evict_select_kernel, total_dev, total_ld, len_dev, max_len, sinks, recent,
                                    budget, slice, cached, keep_dev, keep_ld, new_len_dev, status_dev));
    return NSA_OK;
}

extern "C" size_t nsa_evict_compact_workspace_bytes(int B, int max_len)
{
    if (B <= 0 || max_len <= 0) return 0;
    return 16 + (size_t)B * (size_t)nsa::ceil_div(max_len, nsa::kCpMinT) * sizeof(int32_t);
}

extern "C" nsa_status nsa_evict_compact(int B, const int32_t *keep_dev, int64_t keep_ld, int budget,
                                        const int32_t *new_len_dev, const int32_t *old_len_dev, int max_len,
                                        const int32_t *page_table_dev, int64_t pt_ld, int page_size, int64_t num_pages,
                                        int n_arrays, void *const *arrays_dev, const int64_t *row_bytes,
                                        float *total_dev, int64_t total_ld, void *workspace_dev,
                                        size_t workspace_bytes, int32_t *status_dev, nsa_stream_t stream)
{
    using namespace nsa;
    if (B < 0 || max_len < 0 || budget < 0 || keep_ld < budget || page_size < 1 || num_pages < 0 || n_arrays < 0 ||
        n_arrays > kMaxArrays || pt_ld < ceil_div(max_len, page_size))
        return NSA_ERR_INVALID_ARG;
    if (n_arrays > 0 && (!arrays_dev || !row_bytes)) return NSA_ERR_INVALID_ARG;
    if (total_dev && total_ld < max_len) return NSA_ERR_INVALID_ARG;
    if (max_len > (1 << 30) || num_pages > 2147483647LL / page_size) return NSA_ERR_UNSUPPORTED;
    CompactParams p = {};
    int64_t row = 0;
    for (int a = 0; a < n_arrays; ++a) {
        if (row_bytes[a] < 1) return NSA_ERR_INVALID_ARG;
        if (row_bytes[a] > kCpMaxRow) return NSA_ERR_UNSUPPORTED;
        row += ceil_div(row_bytes[a], 16) * 16;  // at most what the array's part of the stage takes per position
    }
    if (row > kCpMaxRow) return NSA_ERR_UNSUPPORTED;
    if (B == 0 || max_len == 0 || (n_arrays == 0 && !total_dev)) return NSA_OK;
    if (!keep_dev || !new_len_dev || !old_len_dev || !page_table_dev || num_pages < 1) return NSA_ERR_INVALID_ARG;
    if (((uintptr_t)keep_dev | (uintptr_t)new_len_dev | (uintptr_t)old_len_dev | (uintptr_t)page_table_dev |
         (uintptr_t)total_dev | (uintptr_t)status_dev) & 3)
        return NSA_ERR_INVALID_ARG;
    const size_t need = nsa_evict_compact_workspace_bytes(B, max_len);
    if (!workspace_dev || workspace_bytes < need || ((uintptr_t)workspace_dev & 15)) return NSA_ERR_INVALID_ARG;
    p.T = kCpMaxT;
    while (p.T > kCpMinT && p.T * row > kCpStage) p.T /= 2;
    int64_t stage = 0;
    for (int a = 0; a < n_arrays; ++a) {
        if (!arrays_dev[a]) return NSA_ERR_INVALID_ARG;
        p.array[a] = (uint8_t *)arrays_dev[a];
        p.row_bytes[a] = (int)row_bytes[a];
        const uintptr_t both = (uintptr_t)arrays_dev[a] | (uintptr_t)row_bytes[a];
        p.unit[a] = both % 16 == 0 ? 16 : both % 4 == 0 ? 4 : 1;
        p.offset[a] = (int)stage;
        stage += ceil_div(p.T * row_bytes[a], 16) * 16;
    }
    p.n_arrays = n_arrays;
    p.keep = keep_dev; p.keep_ld = keep_ld;
    p.new_len = new_len_dev; p.old_len = old_len_dev;
    p.page_table = page_table_dev; p.pt_ld = pt_ld; p.page_size = page_size; p.num_pages = num_pages;
    p.max_len = max_len; p.budget = budget;
    p.total = total_dev; p.total_ld = total_ld;
    p.chunks = (int)ceil_div(max_len, p.T); p.B = B;
    if ((int64_t)B * p.chunks > 0x7fffffffLL - 0x100000) return NSA_ERR_UNSUPPORTED;
    p.ticket = (int32_t *)workspace_dev;
    p.read_done = p.ticket + 4;
    p.status = status_dev;
    const int sms = current_sm_count();
    if (sms <= 0) return NSA_ERR_CUDA;
    const cudaStream_t s = (cudaStream_t)stream;
    NSA_CUDA_TRY(cudaMemsetAsync(workspace_dev, 0, 16 + (size_t)B * p.chunks * sizeof(int32_t), s));
    NSA_CUDA_TRY(cudaFuncSetAttribute(evict_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      kCpMinT * kCpMaxRow));
    const int64_t tickets = (int64_t)B * p.chunks, most = (int64_t)sms * 4;
    evict_compact_kernel<<<(unsigned)(tickets < most ? tickets : most), kCpThreads, (size_t)stage, s>>>(p);
    return launch_status();
}
