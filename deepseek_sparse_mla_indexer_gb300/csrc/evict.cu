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
#include "sm100_paged.cuh"

namespace nsa {
namespace {

using namespace sm100;

// ------------------------------------------------------------------ select
//
// One thread-block cluster per request; its CTAs own equal slices of the
// positions and its warps contiguous parts of them, a key per lane and step.  The
// threshold key of the middle range is found by a radix selection over 11 + 11 +
// 10 bits of the order-preserving key.  Pass 0 counts the leading digits of all
// keys in shared memory; after a cluster barrier every CTA sums the counts of all
// (distributed shared memory) and finds the same digit.  The keys with that digit,
// some per cent of them, go into a list in shared memory, from which passes 1 and 2
// count; where they do not fit (totals that are mostly equal) the passes run over
// all keys again.  Then every CTA writes its kept positions behind those of the
// CTAs before it: positions above the threshold, and of those equal to it the
// lowest ones.  Keys stay in shared memory (slices up to 40 K; longer ones are read
// again from L2).  Whole numbers throughout: the result does not depend on
// scheduling.  Not bound by its bytes: 31 us for 16 requests of 50000 .. 131072 totals
// (7.5 MB), whose 64 CTAs leave 88 SMs idle and walk 32 keys a thread four times between a
// dozen barriers.  One request of 4099 takes 14 - 17 us, the host's part of a call; 8 us in a graph.
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelMaxCluster = 8;         // the portable limit
constexpr int kSelSlice = 16 * 1024;      // positions a CTA takes while the clusters run in one wave
constexpr int kSelCache = 40 * 1024;      // keys that fit in shared memory
constexpr int kSelList = 2048;

struct SelShared {
    alignas(16) uint32_t hist[3][2048];    // one per pass: none is cleared while a peer may read it
    uint32_t list[kSelList];               // keys that share the threshold's first digit
    uint32_t scan[kSelWarps];
    uint32_t digit, need, listed;
    uint32_t warp_sure[kSelWarps], warp_eq[kSelWarps];
    uint32_t cta_sure, cta_eq;             // this CTA's counts, read by the others
};

__device__ __forceinline__ uint32_t dsmem_ld_u32(const uint32_t *local, uint32_t rank)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(dsmem_addr(local, rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint2 dsmem_ld_u32x2(const uint32_t *local, uint32_t rank)
{
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(dsmem_addr(local, rank)) : "memory");
    return v;
}

// Adds 1 to hist[bin] for every lane with `on`; a warp whose lanes all name one
// bin (rows of equal totals) adds once.
__device__ __forceinline__ void count_digit(uint32_t *hist, uint32_t bin, bool on, int lane)
{
    const uint32_t first = __shfl_sync(0xffffffffu, bin, 0);
    if (__all_sync(0xffffffffu, on && bin == first)) {
        if (lane == 0) atomicAdd(hist + bin, 32u);
    } else if (on) {
        atomicAdd(hist + bin, 1u);
    }
}

// CACHED: the slice's keys are kept in shared memory, [slice rounded up to 1024].
template <bool CACHED>
__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const float *total, int64_t total_ld, const int32_t *lens, int max_len, int sinks, int recent,
                    int budget, int slice, int32_t *keep, int64_t keep_ld, int32_t *new_len, int32_t *status)
{
    extern __shared__ uint32_t key_s[];
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
    // this warp's part: steps of 32 consecutive positions; lane's position and key of step j
    const int steps = (p1 - p0 + kSelThreads - 1) / kSelThreads;
    const int w0 = p0 + warp * steps * 32 + lane;
    uint32_t *mine = key_s + warp * steps * 32 + lane;
    auto in_mid = [&](int pos) { return pos < p1 && pos >= mid0 && pos < mid1; };
    auto sync_cluster = [&]() {
        if (nc > 1)
            cluster_sync_all();
        else
            __syncthreads();
    };
    auto key_at = [&](int j) -> uint32_t {
        return CACHED ? mine[32 * j] : in_mid(w0 + 32 * j) ? order_key(__ldg(row + w0 + 32 * j)) : 0u;
    };
    for (int i = tid; i < 3 * 2048 / 4; i += kSelThreads) reinterpret_cast<uint4 *>(sm.hist)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) sm.listed = 0;
    __syncthreads();

    uint32_t need = (uint32_t)(budget - sinks - recent), prefix = 0;
    const bool any = need > 0;  // else nothing between the ends is kept
    if (any) {
        constexpr int kAhead = 8;  // loads in flight a thread
        for (int j0 = 0; j0 < steps; j0 += kAhead) {
            float v[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int pos = w0 + 32 * (j0 + u);
                v[u] = j0 + u < steps && in_mid(pos) ? __ldg(row + pos) : 0.f;
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (j0 + u >= steps) break;
                const bool on = in_mid(w0 + 32 * (j0 + u));
                const uint32_t k = on ? order_key(v[u]) : 0u;
                if (CACHED) mine[32 * (j0 + u)] = k;
                count_digit(sm.hist[0], k >> 21, on, lane);
            }
        }
        bool listed = false;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            uint32_t *hist = sm.hist[pass];
            if (pass > 0) {
                const int shift = pass == 1 ? 10 : 0, above_shift = pass == 1 ? 21 : 10;
                const uint32_t mask = pass == 1 ? 2047u : 1023u;
                if (pass == 1) {
                    // the keys of the threshold's first digit into the list
#pragma unroll 4
                    for (int j = 0; j < steps; ++j) {
                        const uint32_t k = key_at(j);
                        const bool on = (k >> 21) == prefix && in_mid(w0 + 32 * j);
                        const uint32_t who = __ballot_sync(0xffffffffu, on);
                        if (who) {
                            uint32_t at = 0;
                            if (lane == 0) at = atomicAdd(&sm.listed, (uint32_t)__popc(who));
                            at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1u));
                            if (on && at < kSelList) sm.list[at] = k;
                        }
                    }
                    __syncthreads();
                    listed = sm.listed <= kSelList;
                }
                if (listed) {
                    for (uint32_t i = tid; i < sm.listed; i += kSelThreads) {
                        const uint32_t k = sm.list[i];
                        if ((k >> above_shift) == prefix) atomicAdd(hist + ((k >> shift) & mask), 1u);
                    }
                } else {
                    for (int j = 0; j < steps; ++j) {
                        const uint32_t k = key_at(j);
                        const bool on = (k >> above_shift) == prefix && in_mid(w0 + 32 * j);
                        if (__any_sync(0xffffffffu, on)) count_digit(hist, (k >> shift) & mask, on, lane);
                    }
                }
            }
            sync_cluster();  // every CTA's counts are complete
            // bins 2 tid, 2 tid + 1 over the cluster, then counts from the top
            uint2 c = make_uint2(0u, 0u);
            for (int q = 0; q < nc; ++q) {
                const uint2 v = dsmem_ld_u32x2(hist + 2 * tid, (uint32_t)q);
                c.x += v.x;
                c.y += v.y;
            }
            uint32_t suf = c.x + c.y;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_down_sync(0xffffffffu, suf, o);
                if (lane + o < 32) suf += v;
            }
            if (lane == 0) sm.scan[warp] = suf;
            __syncthreads();
            uint32_t above = lane > warp ? sm.scan[lane] : 0u;
            above = __reduce_add_sync(0xffffffffu, above) + suf - (c.x + c.y);
            // the bin where the count from the top reaches `need`: exactly one thread has it
            if (above < need && above + c.y >= need) {
                sm.digit = 2 * tid + 1;
                sm.need = need - above;
            } else if (above + c.y < need && above + c.y + c.x >= need) {
                sm.digit = 2 * tid;
                sm.need = need - above - c.y;
            }
            __syncthreads();
            prefix = (prefix << (pass == 2 ? 10 : 11)) | sm.digit;
            need = sm.need;
        }
    }
    const uint32_t threshold = prefix;
    auto classify = [&](int j, bool &sure, bool &eq) {
        const int pos = w0 + 32 * j;
        const bool mid = in_mid(pos);
        const uint32_t k = any ? key_at(j) : 0u;
        sure = pos < p1 && (!mid || (any && k > threshold));
        eq = mid && any && k == threshold;
    };
    uint32_t n_sure = 0, n_eq = 0;
#pragma unroll 4
    for (int j = 0; j < steps; ++j) {
        bool sure, eq;
        classify(j, sure, eq);
        n_sure += sure;
        n_eq += eq;
    }
    n_sure = __reduce_add_sync(0xffffffffu, n_sure);
    n_eq = __reduce_add_sync(0xffffffffu, n_eq);
    if (lane == 0) {
        sm.warp_sure[warp] = n_sure;
        sm.warp_eq[warp] = n_eq;
    }
    __syncthreads();
    const uint32_t ws = sm.warp_sure[lane], we = sm.warp_eq[lane];
    uint32_t sure_before = __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0u);
    uint32_t eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? we : 0u);
    if (nc > 1) {
        if (warp == 0) {
            const uint32_t all_sure = __reduce_add_sync(0xffffffffu, ws), all_eq = __reduce_add_sync(0xffffffffu, we);
            if (lane == 0) {
                sm.cta_sure = all_sure;
                sm.cta_eq = all_eq;
            }
        }
        cluster_sync_all();
        const uint32_t cs = lane < rank ? dsmem_ld_u32(&sm.cta_sure, (uint32_t)lane) : 0u;
        const uint32_t ce = lane < rank ? dsmem_ld_u32(&sm.cta_eq, (uint32_t)lane) : 0u;
        sure_before += __reduce_add_sync(0xffffffffu, cs);
        eq_before += __reduce_add_sync(0xffffffffu, ce);
    }
    // a position's place: the sure ones before it plus the equal ones taken before it
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
    for (int j = 0; j < steps; ++j) {
        bool sure, eq;
        classify(j, sure, eq);
        const uint32_t bs = __ballot_sync(0xffffffffu, sure), be = __ballot_sync(0xffffffffu, eq);
        const uint32_t e = eq_before + __popc(be & below);
        if (sure || (eq && e < need)) out[sure_before + __popc(bs & below) + min(e, need)] = w0 + 32 * j;
        eq_before += __popc(be);
        sure_before += __popc(bs);
    }
    if (rank == 0 && tid == 0) new_len[b] = budget;
    if (nc > 1) cluster_sync_all();  // a peer may still read this CTA's counts
}

// Clusters of nc selection CTAs that the current device runs at once (asked once per device).
int select_clusters(int nc)
{
    constexpr int kMaxDev = 64;
    static std::atomic<int> cache[kMaxDev][kSelMaxCluster + 1];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDev) return 1;
    n = cache[dev][nc].load(std::memory_order_relaxed);
    if (n > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)nc);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = kSelSlice * 4;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)nc;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (max_dynamic_smem<evict_select_kernel<true>>(kSelCache * 4) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, evict_select_kernel<true>, &cfg) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();  // a failed query is not the caller's error
        n = 1;
    }
    cache[dev][nc].store(n, std::memory_order_relaxed);
    return n;
}

// ------------------------------------------------------------------ compact
//
// Position i of a request's front takes the row of position keep[i], in place.
// keep ascends, so keep[i] >= i: rows only move towards the front, and a row
// may be overwritten as soon as it has been read.  The kept positions are cut into
// chunks of T; a CTA stages its chunk's source rows in shared memory, announces
// that it has read them, waits until every chunk that reads rows from its own
// destination range has announced the same, and writes.  Those are chunks with
// lower numbers (keep[j] >= j), at most two besides itself (each spans at least
// T source positions).  The totals behind the kept positions are cleared by chunks
// of kCpTail positions under the same rule.  Chunks are handed out in ascending
// order, the clearing ones last, so the waits end: a CTA waits only for chunks that
// were handed out before its own, and the lowest unfinished one never waits.
//
// Bound by HBM: every row that moves is read and written once; rows that stay are
// not touched.  A chunk is a chain of dependent loads (ticket, lengths, kept
// positions, pages, rows).  Four warps walk it for the CTA's next chunk while the
// other four move the current one, whose rows go through shared memory as bulk
// copies (a thread issues one copy a row and array), and several CTAs share an SM.
// Measured (GB300): 4 requests of 65536 .. 131072 positions cut to 50000, bf16 rows, indexer keys
// and scales (518 MB moved): 105 us, 4.9 TB/s, 73 % of the copy rate; 32 requests of 4096 .. 32768
// cut to 5001, fp8 rows (232 MB): 57 us, 60 %; one of 4099: 16 us (12 in a graph).
constexpr int kMaxArrays = 8;
constexpr int kCpThreads = 256;          // warps 0..3 move a chunk, warps 4..7 describe the next one
constexpr int kMovers = 128;
constexpr int kCpMinT = 8, kCpMaxT = 128;
constexpr int kCpTail = 4096;            // totals cleared by one chunk
constexpr int kCpStage = 52 * 1024;      // bytes staged per CTA at most, where a chunk of kCpMinT allows it
constexpr int kCpPerSm = 8;              // CTAs per SM at most
constexpr int kCpMaxRow = 24 * 1024;     // bytes of one position over all arrays
constexpr long long kCpWait = 2000000000LL;  // ~1 s of SM clocks

struct CompactParams {
    uint8_t *array[kMaxArrays];
    int row_bytes[kMaxArrays];
    int unit[kMaxArrays];       // bytes per copy step: 16, 4 or 1
    uint32_t per[kMaxArrays];   // steps per row
    uint32_t magic[kMaxArrays]; // ceil(2^32 / per): step / per is its high product; 0: divide
    int offset[kMaxArrays];     // of the array's rows within the stage
    int n_arrays;
    int bulk_bytes;             // bytes of a position in the arrays of unit 16
    const int32_t *keep;
    int64_t keep_ld;
    const int32_t *new_len, *old_len;
    const int32_t *page_table;
    int64_t pt_ld;
    int page_size, max_len, budget;
    int64_t num_pages;
    float *total;
    int64_t total_ld;
    int T, chunks, tails, B;    // per request: chunks of T kept positions, tails of kCpTail positions
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

// The number of entries of the ascending keep[0 .. n) below `v`, by one warp.
__device__ __forceinline__ int warp_lower_bound(const int32_t *keep, int n, int v, int lane)
{
    int lo = 0, len = n;  // the answer lies in [lo, lo + len]
    while (len > 0) {
        const int step = (len + 31) / 32;
        const int i = lane * step;
        const int c = __popc(__ballot_sync(0xffffffffu, i < len && keep[lo + i] < v));
        if (c == 0) return lo;
        if (step == 1) return lo + c;
        lo += (c - 1) * step + 1;  // entry (c - 1) * step is below v
        len = min(step - 1, len - (c - 1) * step - 1);
    }
    return lo;
}

// What a CTA knows of a chunk before it moves its rows.
struct Chunk {
    int32_t src[kCpMaxT], dst[kCpMaxT];  // slots; -1: the row does not move
    int32_t from[kCpMaxT];               // position whose total moves here, -1: cleared, -2: not of this chunk
    int ticket, b, c;                    // c < 0: tail chunk -c - 1
    int lo, hi;                          // destination positions
    int w0, w1;                          // chunks w0 .. w1-1 read from there
    int run;                             // 0: nothing to do
    int moving;                          // rows that move
};

// The chunk of `ticket`, by warps 4..7: two walk the rows, two look for the chunks to wait for.
__device__ __forceinline__ void describe(const CompactParams &p, Chunk &k, int ticket)
{
    const int warp = (threadIdx.x >> 5) - 4, lane = threadIdx.x & 31;
    // tickets go round the requests first: a chunk's predecessors are then well ahead of it
    const int rows = p.B * p.chunks;
    const bool tail = ticket >= rows;
    const int x = tail ? ticket - rows : ticket;
    const int c = x / p.B, b = x - c * p.B;
    const int old = p.old_len[b], n = p.new_len[b];
    const bool bad = old < 0 || old > p.max_len || n < 0 || n > old || n > p.budget;
    const int lo = tail ? max(n, c * kCpTail) : c * p.T;
    const int hi = tail ? min(old, (c + 1) * kCpTail) : min(n, lo + p.T);
    const bool run = !bad && n < old && lo < hi && (!tail || p.total);
    const int32_t *keep = p.keep + (int64_t)b * p.keep_ld;
    if (warp < 2) {
        const int32_t *pt = p.page_table + (int64_t)b * p.pt_ld;
        for (int r = warp * 32 + lane; r < p.T; r += 64) {
            int32_t s = -1, d = -1, from = -2;
            const int i = lo + r;
            if (run && !tail && i < hi) {
                const int q = keep[i], before = i > 0 ? keep[i - 1] : -1;
                from = q;
                if (q < i || q >= old || before >= q) {
                    set_status(p.status, NSA_ERR_BOUNDS);  // not an ascending list of positions: likewise
                    from = i;
                } else if (q != i && p.n_arrays > 0) {
                    const int sp = q / p.page_size, dp = i / p.page_size;
                    const int32_t ps = pt[sp], pd = pt[dp];
                    if (ps < 0 || ps >= p.num_pages || pd < 0 || pd >= p.num_pages) {
                        set_status(p.status, NSA_ERR_BOUNDS);  // a page outside the cache: the row stays, and its total
                        from = i;
                    } else {
                        s = ps * p.page_size + (q - sp * p.page_size);
                        d = pd * p.page_size + (i - dp * p.page_size);
                        atomicAdd(&k.moving, 1);
                    }
                }
            }
            k.src[r] = s;
            k.dst[r] = d;
            k.from[r] = from;
        }
    } else {
        // rows j with lo <= keep[j] < hi are read from the destination range, by chunks j / T
        const bool second = warp == 3;
        const int j = run ? warp_lower_bound(keep, n, second ? hi : lo, lane) : 0;
        if (lane == 0) {
            if (second) {
                k.w1 = (j + p.T - 1) / p.T;
                if (bad && c == 0 && !tail) set_status(p.status, NSA_ERR_BOUNDS);
            } else {
                k.w0 = j / p.T;
                k.b = b;
                k.c = tail ? -c - 1 : c;
                k.lo = lo;
                k.hi = hi;
                k.run = run ? 1 : 0;
            }
        }
    }
}

template <int UNIT> struct CopyUnit;
template <> struct CopyUnit<4> { using type = uint32_t; };
template <> struct CopyUnit<1> { using type = uint8_t; };

// Rows of one array of 4-byte or odd rows between the cache and the stage.
template <int UNIT, bool READ>
__device__ __forceinline__ void move_rows(uint8_t *array, int row_bytes, uint32_t per, uint32_t magic, uint8_t *stage,
                                          const int32_t *slot, int T)
{
    using U = typename CopyUnit<UNIT>::type;
    for (uint32_t e = threadIdx.x; e < T * per; e += kMovers) {
        const uint32_t i = magic ? __umulhi(e, magic) : e / per, c = e - i * per;
        const int64_t at = slot[i];
        if (at < 0) continue;
        U *g = reinterpret_cast<U *>(array + at * row_bytes) + c;
        U *s = reinterpret_cast<U *>(stage) + e;  // rows of the stage follow one another
        if constexpr (READ && UNIT == 4)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(s)), "l"(g) : "memory");
        else if constexpr (READ)
            *s = __ldcg(g);
        else
            *g = *s;
    }
}

// Every array's rows of the chunk, by the movers.
template <bool READ>
__device__ __forceinline__ void move_all(const CompactParams &p, uint8_t *stage, const int32_t *slot, uint64_t *bar)
{
    if (threadIdx.x < (unsigned)p.T) {
        const int64_t at = slot[threadIdx.x];
        if (at >= 0)
            for (int a = 0; a < p.n_arrays; ++a) {
                if (p.unit[a] != 16) continue;
                uint8_t *g = p.array[a] + at * p.row_bytes[a], *s = stage + p.offset[a] + threadIdx.x * p.row_bytes[a];
                if (READ)
                    bulk_load(s, g, (uint32_t)p.row_bytes[a], bar);
                else
                    bulk_store(g, s, (uint32_t)p.row_bytes[a]);
            }
        if (!READ) bulk_commit();
    }
    for (int a = 0; a < p.n_arrays; ++a) {
        if (p.unit[a] == 4)
            move_rows<4, READ>(p.array[a], p.row_bytes[a], p.per[a], p.magic[a], stage + p.offset[a], slot, p.T);
        else if (p.unit[a] == 1)
            move_rows<1, READ>(p.array[a], p.row_bytes[a], p.per[a], p.magic[a], stage + p.offset[a], slot, p.T);
    }
}

__global__ void __launch_bounds__(kCpThreads) evict_compact_kernel(CompactParams p)
{
    extern __shared__ __align__(16) uint8_t stage[];
    __shared__ Chunk chunk[2];
    __shared__ uint64_t landed;
    __shared__ int next_ticket[2], timed_out;  // by parity: one is read while the other is drawn
    const int tid = threadIdx.x;
    const bool mover = tid < kMovers;
    const int n_tickets = p.B * (p.chunks + p.tails);
    if (tid == 0) {
        mbar_init(&landed, 1);
        fence_mbar_init();
        timed_out = 0;
        chunk[0].moving = chunk[1].moving = 0;
        next_ticket[0] = atomicAdd(p.ticket, 1);
    }
    __syncthreads();
    int ticket = next_ticket[0];
    if (!mover && ticket < n_tickets) describe(p, chunk[0], ticket);
    __syncthreads();
    uint32_t phase = 0;
    for (int it = 0; ticket < n_tickets; ++it) {
        Chunk &k = chunk[it & 1], &next = chunk[(it + 1) & 1];
        // a ticket held while this chunk is worked on: it is higher than this one, so no wait on it is circular
        if (tid == kMovers) {
            next_ticket[(it + 1) & 1] = atomicAdd(p.ticket, 1);
            next.moving = 0;
        }
        if (!mover) {
            bar_sync(2, kCpThreads - kMovers);
            const int drawn = next_ticket[(it + 1) & 1];
            if (drawn < n_tickets) describe(p, next, drawn);  // while the rows of this chunk move
        } else if (k.run) {
            float t = 0.f;
            float *total = p.total ? p.total + (int64_t)k.b * p.total_ld : nullptr;
            if (k.c >= 0) {
                if (tid == 0) mbar_arrive_expect_tx(&landed, (uint32_t)(k.moving * p.bulk_bytes));
                move_all<true>(p, stage, k.src, &landed);
                if (total && tid < p.T && k.from[tid] >= 0) t = __ldcg(total + k.from[tid]);
                cp_async_commit();
                cp_async_wait_all();
                if (!mbar_wait(&landed, phase, kCpWait)) {
                    set_status(p.status, NSA_ERR_TIMEOUT);
                    timed_out = 1;
                }
                phase ^= 1;
            }
            bar_sync(1, kMovers);  // every mover's reads (rows and totals) have arrived
            int32_t *done = p.read_done + (int64_t)k.b * p.chunks;
            if (tid == 0 && k.c >= 0) st_release(done + k.c, 1);
            const int w1 = k.c >= 0 ? min(k.w1, k.c) : k.w1;  // later chunks read behind this one's destination
            for (int x = k.w0 + tid; x < w1; x += kMovers) {
                const long long t0 = clock64();
                while (!ld_acquire(done + x)) {
                    if (clock64() - t0 > kCpWait) {
                        set_status(p.status, NSA_ERR_TIMEOUT);
                        timed_out = 1;
                        break;
                    }
                    __nanosleep(32);
                }
            }
            bar_sync(1, kMovers);
            if (!timed_out) {  // else rows that another chunk may not have read are left as they are
                if (k.c >= 0) {
                    move_all<false>(p, stage, k.dst, nullptr);
                    if (total && tid < p.T && k.from[tid] >= 0) total[k.lo + tid] = t;
                } else {
                    for (int i = k.lo + tid; i < k.hi; i += kMovers) total[i] = 0.f;
                }
            }
        }
        if (mover) bulk_wait_read();  // the rows written last have left the stage
        __syncthreads();              // and the next chunk is described
        ticket = next_ticket[(it + 1) & 1];
        if (timed_out) break;
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
    // CTAs for slices of 16 K; half as many, of 32 K, where the clusters of all requests then run in one
    // wave and did not before (16 x 131072 positions: 8 CTAs of 16 K took two waves of 21 us)
    int nc = 1;
    while (nc < kSelMaxCluster && (int64_t)nc * kSelSlice < max_len) nc *= 2;
    if (nc > 1 && B > select_clusters(nc) && (int64_t)nc * kSelSlice >= max_len) nc /= 2;
    if ((int64_t)B * nc > 0x7fffffffLL) return NSA_ERR_UNSUPPORTED;
    const int slice = max_len > 0 ? (int)ceil_div(max_len, nc) : 1;
    const int cache = (int)ceil_div(slice, kSelThreads) * kSelThreads;
    const bool cached = cache <= kSelCache;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * nc));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = cached ? (size_t)cache * 4 : 0;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)nc;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cached) NSA_CUDA_TRY(max_dynamic_smem<evict_select_kernel<true>>(kSelCache * 4));
    NSA_CUDA_TRY(cudaLaunchKernelEx(&cfg, cached ? evict_select_kernel<true> : evict_select_kernel<false>, total_dev,
                                    total_ld, len_dev, max_len, sinks, recent, budget, slice, keep_dev, keep_ld,
                                    new_len_dev, status_dev));
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
        if (p.unit[a] == 16) p.bulk_bytes += p.row_bytes[a];
        p.per[a] = (uint32_t)(row_bytes[a] / p.unit[a]);
        // exact while step * per < 2^32, which short rows keep (at most kCpMinT * kCpMaxRow steps)
        p.magic[a] = p.per[a] > 1 && p.per[a] < 4096 ? (uint32_t)((0x100000000ULL + p.per[a] - 1) / p.per[a]) : 0;
        p.offset[a] = (int)stage;
        stage += ceil_div(p.T * row_bytes[a], 16) * 16;
    }
    p.n_arrays = n_arrays;
    p.keep = keep_dev; p.keep_ld = keep_ld;
    p.new_len = new_len_dev; p.old_len = old_len_dev;
    p.page_table = page_table_dev; p.pt_ld = pt_ld; p.page_size = page_size; p.num_pages = num_pages;
    p.max_len = max_len; p.budget = budget;
    p.total = total_dev; p.total_ld = total_ld;
    p.chunks = (int)ceil_div(budget < max_len ? budget : max_len, p.T);
    p.tails = total_dev ? (int)ceil_div(max_len, kCpTail) : 0;
    p.B = B;
    const int64_t tickets = (int64_t)B * (p.chunks + p.tails);
    if (tickets > 0x7fffffffLL - 0x100000) return NSA_ERR_UNSUPPORTED;
    if (tickets == 0) return NSA_OK;
    p.ticket = (int32_t *)workspace_dev;
    p.read_done = p.ticket + 4;
    p.status = status_dev;
    const int sms = current_sm_count();
    if (sms <= 0) return NSA_ERR_CUDA;
    const cudaStream_t s = (cudaStream_t)stream;
    NSA_CUDA_TRY(cudaMemsetAsync(workspace_dev, 0, 16 + (size_t)B * p.chunks * sizeof(int32_t), s));
    NSA_CUDA_TRY(max_dynamic_smem<evict_compact_kernel>(kCpMinT * kCpMaxRow));
    const int64_t fit = (227 * 1024) / (stage + (int64_t)sizeof(Chunk) * 2 + 2048);  // by shared memory
    const int64_t most = (int64_t)sms * (fit < 1 ? 1 : fit < kCpPerSm ? fit : kCpPerSm);
    evict_compact_kernel<<<(unsigned)(tickets < most ? tickets : most), kCpThreads, (size_t)stage, s>>>(p);
    return launch_status();
}
