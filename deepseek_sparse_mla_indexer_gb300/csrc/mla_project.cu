// The products with the key/value up-projection w [H * 256, 512] (bf16), whose rows are, for each
// head, 128 rows W_k that give keys from latents and 128 rows W_v that give values:
//   nsa_mla_expand_kv   kv[t, h, :]  = w[h] c_t        (256 x 512; c_t gathered from the paged cache)
//   nsa_mla_absorb_q    out[r, h, :] = q[r, h] W_k[h]  (128 -> 512)
//   nsa_mla_project_v   out[r, h, :] = W_v[h] c[r, h]  (512 -> 128)
//
// One tcgen05 kernel: D[128 features, N rows] = W_tile . X_tile^T with W as the operand of 128 rows,
// so that a decoding batch of R rows is a product of N = 16, 32, .. columns that reads each weight
// once, and not one padded to 128 rows.  absorb's weights are contiguous along the features (an
// MN-major operand), the others' along the product's axis.  Tiles come by TMA in steps of 64 along
// the product's axis through a ring of as many stages as shared memory holds; the accumulators are
// double-buffered in TMEM, so that eight warps turn one tile into bf16 rows, staged in shared memory
// and stored by TMA (which leaves out what lies behind the last row), under the products of the next.
// Persistent: one CTA an SM walks the tiles.  Sums are fp32, rounded to bf16 once.
//
// Measured (GB300, calls in a graph):
//   expand, 8192 bf16 rows, 128 heads (pairs of CTAs, below)     169 us   1.63 PFLOP/s, 83 % of 1969 TFLOP/s
//   expand, 1037 fp8 rows, 16 heads                                8.7 us, of which the gather is 2.5
//   absorb / project, 32 rows, 128 heads                           4.6 / 4.1 us: 22 MB, mostly weights; the start
//   absorb, 4001 rows, 16 heads                                   15.4 us: 84 MB, 5.5 TB/s; seven rounds of tiles, bound by
//                                                                 what an SM moves between L2 and shared memory
//   project, 4001 rows, 16 heads                                  10.5 us with its 66 MB of input in L2, 15.5 from HBM
// Each launch starts under the end of the one before it and then waits for it (absorb of 4001 rows among other
// calls: 16.8 us, and 18.8 started behind it).
#include "mla_forms.cuh"

namespace nsa {
namespace {

using namespace sm100;

constexpr int kFeat = 128;                     // features of a tile
constexpr int kStep = 64;                      // of the product's axis: a 128-byte row of the operands
constexpr uint32_t kWStage = kFeat * kStep * 2;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarps + 2);
constexpr int kSmemMax = 227 * 1024;

constexpr int chunk_of(int N) { return N >= 64 ? 32 : 16; }  // rows that a group of four warps stages at a time
constexpr uint32_t x_stage(int N) { return (uint32_t)N * kStep * 2; }
constexpr uint32_t staging_of(int N) { return 2 * 2 * chunk_of(N) * kFeat * 2; }  // two groups, two buffers
constexpr int kMaxStages = 12;
constexpr int stages_of(int N)
{
    const int n = (int)((kSmemMax - 2048 - staging_of(N)) / (kWStage + x_stage(N)));
    return n < kMaxStages ? n : kMaxStages;
}
constexpr uint32_t tmem_cols_of(int N) { return N <= 16 ? 32u : 2u * N; }

struct PShared {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drained;
    uint32_t tmem;
    volatile int abort;
};
static_assert(sizeof(PShared) <= 1024, "the struct has 1 KB");
constexpr uint32_t smem_of(int N) { return 1024 + stages_of(N) * (kWStage + x_stage(N)) + staging_of(N) + 1024; }

struct PParams {
    int n_ft;          // feature tiles of all heads
    int n_rt;          // row tiles
    int steps;         // of the product's axis
    int ft_per_head;   // feature tiles of a head (of X's rows); expand: all, for one head
    int w_head_rows;   // rows of w a head and its first one
    int w_row0;
    int32_t *status;
};

// ------------------------------------------------------------ accumulators to rows

// 16 lanes x 8 CH / 8 columns of the warp's 32 lanes: thread i gets lanes i / 4 and i / 4 + 8, of every eight
// columns 2 (i % 4) and the one behind it (registers 4 b .. 4 b + 3 of columns 8 b ..).
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// Four 8 x 8 blocks of 16-bit values, each turned over: a block's columns become the 16-byte rows whose addresses
// lanes 8 b .. 8 b + 7 give.
__device__ __forceinline__ void store_blocks_turned(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// One tile's accumulator (128 features in the lanes, N rows in the columns from `acc` on) as bf16 rows to
// out[row0 ..][head][feat0 ..].  A group of four warps takes every other CH rows: through two staging buffers of
// [2][CH][64 features], 128-byte swizzled so that the turned blocks' rows fall into different banks.
template <int N>
__device__ __forceinline__ void rows_out(const CUtensorMap &out_map, uint32_t acc, uint8_t *stage_s, int &n_store, int feat0,
                                         int head, int row0)
{
    constexpr int CH = chunk_of(N);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, group = warp >> 2, quarter = warp & 3;
    const bool leader = (threadIdx.x & 127) == 0;
    const uint32_t lanes = acc + ((uint32_t)(quarter * 32) << 16);
    for (int k = group; k < N / CH; k += 2, ++n_store) {
        uint8_t *o = stage_s + (group * 2 + (n_store & 1)) * (CH * kFeat * 2);
        uint32_t v[2][CH / 2];
#pragma unroll
        for (int x = 0; x < 2; ++x) tmem_ld_16x256(lanes + ((uint32_t)(16 * x) << 16) + k * CH, v[x]);
        if (leader) bulk_wait_read_1();  // the store before last has read this buffer
        __syncwarp();
        tmem_ld_wait();
        bar_sync(1 + group, 128);
        // blocks of 8 features x 8 rows: lanes 0 .. 7, 8 .. 15 of this half; rows 8 b .., 8 b + 8 ..
        const uint32_t half = smem_u32(o) + (quarter >> 1) * (CH * 128);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int b = 0; b < CH / 8; b += 2) {
                const int r = 8 * b + (lane & 7) + (lane >= 16 ? 8 : 0), c16 = (quarter & 1) * 4 + x * 2 + (lane >> 3 & 1);
                const uint32_t *u = &v[x][4 * b];
                store_blocks_turned(half + sw128_offset(r, c16), pack_bf16(__uint_as_float(u[0]), __uint_as_float(u[1])),
                                    pack_bf16(__uint_as_float(u[2]), __uint_as_float(u[3])),
                                    pack_bf16(__uint_as_float(u[4]), __uint_as_float(u[5])),
                                    pack_bf16(__uint_as_float(u[6]), __uint_as_float(u[7])));
            }
        fence_proxy_async_smem();
        bar_sync(1 + group, 128);
        if (leader) {
            tma_store_3d(&out_map, feat0, head, row0 + k * CH, o);
            tma_store_3d(&out_map, feat0 + 64, head, row0 + k * CH, o + CH * 128);
            bulk_commit();
        }
        __syncwarp();
    }
}

// MN_W: W_k, whose tile of 128 features x 64 is two boxes of 64 features, [64][64 features].
template <int N, bool MN_W>
__global__ void __launch_bounds__(kThreads, 1)
head_product_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map,
                    const __grid_constant__ CUtensorMap out_map, PParams p)
{
    constexpr int ST = stages_of(N);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *w_s = base, *x_s = w_s + ST * kWStage, *stage_s = x_s + ST * x_stage(N);
    PShared *sm = (PShared *)(stage_s + staging_of(N));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&sm->full[i], 1);
            mbar_init(&sm->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm->acc_full[i], 1);
            mbar_init(&sm->acc_empty[i], kEpiWarps);
        }
        mbar_init(&sm->drained, 1);
        sm->abort = 0;
        fence_mbar_init();
        prefetch_tensormap(&w_map);
        prefetch_tensormap(&x_map);
        prefetch_tensormap(&out_map);
    }
    if (warp == kEpiWarps) tmem_alloc(&sm->tmem, tmem_cols_of(N));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm->tmem;
    const int tiles = p.n_ft * p.n_rt;  // at most 2^30 (the launch checks)
    // The launch before this one may still run (its last blocks leave room for this one's start).  Every warp waits for
    // its end here, so that none of the bounded waits below counts its time
    pdl_wait();

    if (warp == kEpiWarps) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            int st = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const int rt = t / p.n_ft, ft = t - rt * p.n_ft;
                const int h = ft / p.ft_per_head, c = ft - h * p.ft_per_head;
                const int w_row = h * p.w_head_rows + p.w_row0;
                for (int s = 0; s < p.steps; ++s) {
                    if (!(ok = mla_wait(&sm->empty[st], ph ^ 1, &sm->abort))) break;
                    mbar_arrive_expect_tx(&sm->full[st], kWStage + x_stage(N));
                    uint8_t *w = w_s + st * kWStage;
                    if (MN_W) {
                        tma_load_2d(w, &w_map, c * kFeat, w_row + s * kStep, &sm->full[st]);
                        tma_load_2d(w + kWStage / 2, &w_map, c * kFeat + 64, w_row + s * kStep, &sm->full[st]);
                    } else {
                        tma_load_2d(w, &w_map, s * kStep, w_row + c * kFeat, &sm->full[st]);
                    }
                    tma_load_3d(x_s + st * x_stage(N), &x_map, s * kStep, h, rt * N, &sm->full[st]);
                    if (++st == ST) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            }
            if (!ok) {
                set_status(p.status, NSA_ERR_TIMEOUT);
                // copies in flight end before the block does: stages before st were filled last with phase ph
                for (int i = 0; i < ST; ++i) mbar_wait(&sm->full[i], i < st ? ph : ph ^ 1, kMlaWait);
            }
        }
        __syncwarp();
    } else if (warp == kEpiWarps + 1) {
        // ------------------------------------------------------------ products
        const uint32_t idesc = instr_desc(1, 1, MN_W ? 1 : 0, 0, kFeat, N);
        const uint64_t w_desc = MN_W ? smem_desc(smem_u32(w_s), kWStage / 2, 1024, kSwizzle128B)
                                     : smem_desc(smem_u32(w_s), 16, 1024, kSwizzle128B);
        const uint64_t x_desc = smem_desc(smem_u32(x_s), 16, 1024, kSwizzle128B);
        int st = 0, i = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++i) {
            const uint32_t buf = i & 1, bph = (i >> 1) & 1;
            ok = __all_sync(0xffffffffu, mla_wait(&sm->acc_empty[buf], bph ^ 1, &sm->abort));
            tc_fence_after();
            for (int s = 0; s < p.steps && ok; ++s) {
                ok = __all_sync(0xffffffffu, mla_wait(&sm->full[st], ph, &sm->abort));
                tc_fence_after();
                if (ok && elect_one()) {
                    const uint64_t wd = w_desc + st * (kWStage / 16), xd = x_desc + st * (x_stage(N) / 16);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f16(tmem + buf * N, wd + k * (MN_W ? 2048 / 16 : 2), xd + k * 2, idesc, s > 0 || k > 0);
                    mma_commit(&sm->empty[st]);
                    if (s == p.steps - 1) mma_commit(&sm->acc_full[buf]);
                }
                __syncwarp();
                if (++st == ST) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
        if (!ok && lane == 0) {
            set_status(p.status, NSA_ERR_TIMEOUT);
            mma_commit(&sm->drained);  // products in flight end before the block does
            mbar_wait(&sm->drained, 0, kMlaWait);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ rows out
        const int group = warp >> 2;
        const bool leader = (threadIdx.x & 127) == 0;
        int i = 0, n_store = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++i) {
            const int rt = t / p.n_ft, ft = t - rt * p.n_ft;
            const int h = ft / p.ft_per_head, c = ft - h * p.ft_per_head;
            const uint32_t buf = i & 1, bph = (i >> 1) & 1;
            ok = mla_wait(&sm->acc_full[buf], bph, &sm->abort);
            __syncwarp();
            tc_fence_after();
            // the group's warps give up together
            if (bar_red_or(1 + group, 128, !ok)) {
                ok = false;
                break;
            }
            rows_out<N>(out_map, tmem + buf * N, stage_s, n_store, c * kFeat, h, rt * N);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->acc_empty[buf]);
        }
        if (!ok && lane == 0) set_status(p.status, NSA_ERR_TIMEOUT);
        if (leader) bulk_wait_read();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kEpiWarps) {
        tmem_relinquish();
        tmem_dealloc(tmem, tmem_cols_of(N));
    }
}

// ---------------------------------------------------------------- pairs of CTAs

// Large products (nsa_mla_expand_kv of many rows): a 128 x 256 tile a CTA asks L2 for 96 bytes a cycle and SM at
// the tensor core's rate, more than it gives (8192 rows, 128 heads: 203 us, 55 bytes a cycle).  Two CTAs
// (cta_group::2) make a 256 x 256 tile together: each loads 128 rows of W and 128 rows of X, the
// products read the other half of X from the pair's other shared memory, and it is 64.
// CTA 0 issues for both.  CTA 1's loads count on CTA 0's barriers; what CTA 0 has to tell CTA 1 (a stage is free, an
// accumulator is complete) goes from barrier to barrier by a warp of its own.
constexpr int kPairRows = 256;
constexpr uint32_t kPairStage = 2 * kWStage;  // a CTA's 128 rows of W and of X, 64 along the product's axis
constexpr int kPairThreads = 32 * (kEpiWarps + 3);
constexpr int kPairStages = (int)((kSmemMax - 2048 - staging_of(kPairRows)) / kPairStage);
constexpr uint32_t kPairSmem = 1024 + kPairStages * kPairStage + staging_of(kPairRows) + 1024;
static_assert(kPairSmem <= kSmemMax, "shared memory");

struct PairShared {
    uint64_t full[kPairStages], empty[kPairStages], acc_full[2], acc_empty[2], drained;
    uint32_t tmem;
    volatile int abort;
};
static_assert(sizeof(PairShared) <= 1024, "the struct has 1 KB");

// D[tmem of both CTAs] (+)= A B^T, each CTA's half of A and of B at the same place in its shared memory.
__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_commit_pair(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// TMA loads into this CTA that count on a barrier of either CTA of the pair (its address in the cluster).
__device__ __forceinline__ void pair_load_2d(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void pair_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
pair_product_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map,
                    const __grid_constant__ CUtensorMap out_map, PParams p)
{
    constexpr int ST = kPairStages, N = kPairRows;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *w_s = base, *x_s = w_s + ST * kWStage, *stage_s = x_s + ST * kWStage;
    PairShared *sm = (PairShared *)(stage_s + staging_of(N));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = (int)cluster_ctarank();

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&sm->full[i], 1);
            mbar_init(&sm->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm->acc_full[i], 1);
            mbar_init(&sm->acc_empty[i], 2 * kEpiWarps);
        }
        mbar_init(&sm->drained, 1);
        sm->abort = 0;
        fence_mbar_init();
        prefetch_tensormap(&w_map);
        prefetch_tensormap(&x_map);
        prefetch_tensormap(&out_map);
    }
    if (warp == kEpiWarps) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm->tmem)), "r"(512)
                     : "memory");
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();  // barriers of both CTAs before any arrival from the other
    tc_fence_after();
    const uint32_t tmem = sm->tmem;
    const int tiles = p.n_ft * p.n_rt, step = gridDim.x / 2;
    volatile int *abort = &sm->abort;
    bool ok = true;
    pdl_wait();  // every warp, as above

    if (warp == kEpiWarps) {
        // ------------------------------------------------------------ loads of this CTA's halves
        if (lane == 0) {
            int st = 0;
            uint32_t ph = 0;
            for (int t = blockIdx.x / 2; t < tiles && ok; t += step) {
                const int rt = t / p.n_ft, ft = t - rt * p.n_ft;
                for (int s = 0; s < p.steps; ++s) {
                    if (!(ok = mla_wait(&sm->empty[st], ph ^ 1, abort))) break;
                    // CTA 0 expects both CTAs' halves; this stage's next round needs both, so no count runs ahead
                    if (rank == 0) mbar_arrive_expect_tx(&sm->full[st], 2 * kPairStage);
                    const uint32_t bar = dsmem_addr(&sm->full[st], 0);
                    pair_load_2d(w_s + st * kWStage, &w_map, s * kStep, (2 * ft + rank) * kFeat, bar);
                    pair_load_3d(x_s + st * kWStage, &x_map, s * kStep, 0, rt * N + rank * (N / 2), bar);
                    if (++st == ST) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            }
            if (!ok) {
                set_status(p.status, NSA_ERR_TIMEOUT);
                if (rank == 0)
                    for (int i = 0; i < ST; ++i) mbar_wait(&sm->full[i], i < st ? ph : ph ^ 1, kMlaWait);
            }
        }
    } else if (warp == kEpiWarps + 1 && rank == 0) {
        // ------------------------------------------------------------ products of both CTAs
        const uint32_t idesc = instr_desc(1, 1, 0, 0, 2 * kFeat, N);
        const uint64_t w_desc = smem_desc(smem_u32(w_s), 16, 1024, kSwizzle128B);
        const uint64_t x_desc = smem_desc(smem_u32(x_s), 16, 1024, kSwizzle128B);
        int st = 0, i = 0;
        uint32_t ph = 0;
        for (int t = blockIdx.x / 2; t < tiles && ok; t += step, ++i) {
            const uint32_t buf = i & 1, bph = (i >> 1) & 1;
            ok = __all_sync(0xffffffffu, mla_wait(&sm->acc_empty[buf], bph ^ 1, abort));
            for (int s = 0; s < p.steps && ok; ++s) {
                ok = __all_sync(0xffffffffu, mla_wait(&sm->full[st], ph, abort));
                tc_fence_after();
                if (ok && elect_one()) {
                    const uint64_t wd = w_desc + st * (kWStage / 16), xd = x_desc + st * (kWStage / 16);
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_f16_pair(tmem + buf * N, wd + k * 2, xd + k * 2, idesc, s > 0 || k > 0);
                    mma_commit_pair(&sm->empty[st]);
                    if (s == p.steps - 1) mma_commit_pair(&sm->acc_full[buf]);
                }
                __syncwarp();
                if (++st == ST) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
        if (!ok && lane == 0) {
            set_status(p.status, NSA_ERR_TIMEOUT);
            mma_commit_pair(&sm->drained);  // products in flight end before the block does
            mbar_wait(&sm->drained, 0, kMlaWait);
        }
        __syncwarp();
    } else if (warp == kEpiWarps + 2 && rank == 0) {
        // ------------------------------------------------------------ word to the other CTA
        if (lane == 0) {
            int st = 0, i = 0;
            uint32_t ph = 0;
            for (int t = blockIdx.x / 2; t < tiles && ok; t += step, ++i) {
                for (int s = 0; s < p.steps && ok; ++s) {
                    ok = mla_wait(&sm->empty[st], ph, abort);
                    if (ok) mbar_tell(&sm->empty[st], 1);
                    if (++st == ST) {
                        st = 0;
                        ph ^= 1;
                    }
                }
                if (ok) {
                    ok = mla_wait(&sm->acc_full[i & 1], (i >> 1) & 1, abort);
                    if (ok) mbar_tell(&sm->acc_full[i & 1], 1);
                }
            }
            if (!ok) set_status(p.status, NSA_ERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp < kEpiWarps) {
        // ------------------------------------------------------------ rows out
        const int group = warp >> 2;
        const bool leader = (threadIdx.x & 127) == 0;
        int i = 0, n_store = 0;
        for (int t = blockIdx.x / 2; t < tiles; t += step, ++i) {
            const int rt = t / p.n_ft, ft = t - rt * p.n_ft;
            const uint32_t buf = i & 1, bph = (i >> 1) & 1;
            ok = mla_wait(&sm->acc_full[buf], bph, abort);
            __syncwarp();
            tc_fence_after();
            if (bar_red_or(1 + group, 128, !ok)) {
                ok = false;
                break;
            }
            rows_out<N>(out_map, tmem + buf * N, stage_s, n_store, (2 * ft + rank) * kFeat, 0, rt * N);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (rank == 0) mbar_arrive(&sm->acc_empty[buf]);
                else mbar_tell(&sm->acc_empty[buf], 0);
            }
        }
        if (!ok && lane == 0) set_status(p.status, NSA_ERR_TIMEOUT);
        if (leader) bulk_wait_read();
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync_all();  // neither CTA's shared memory or TMEM goes before the other is done with it
    tc_fence_after();
    if (warp == kEpiWarps) {
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

struct Problem {
    const void *w;      // [H * 256, 512]
    const void *x;      // [R, Hx, K] with strides
    int64_t x_ld_r, x_ld_h;
    void *out;          // [R, Ho, F] contiguous
    int H, Hx, R, K, F; // F: features of a head (of Hx)
    int w_head_rows, w_row0;
    bool mn_w, all_heads;  // all_heads: X has none, and all heads' features are one row (expand)
    int32_t *status;
};

// Rows a tile: the width whose waves of tiles take the fewest columns, each tile counted with
// what it costs beside its columns (its 128 x 512 weights take as long as 64 columns of products).
int pick_n(const Problem &q, int sms)
{
    const int64_t n_ft = (int64_t)q.Hx * (q.F / kFeat);
    int best = 256;
    int64_t cost = -1;
    for (int n = 256; n >= 16; n /= 2) {
        const int64_t c = ceil_div(n_ft * ceil_div(q.R, n), sms) * (n + 64);
        if (cost < 0 || c < cost) {
            cost = c;
            best = n;
        }
    }
    return best;
}

template <int N, bool MN_W>
nsa_status launch(const Problem &q, int sms, cudaStream_t stream)
{
    constexpr auto kern = head_product_kernel<N, MN_W>;
    static_assert(smem_of(N) <= kSmemMax, "shared memory");
    CUtensorMap w_map, x_map, out_map;
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const bool mapped =
        make_tma_2d(&w_map, bf, q.w, kMlaLatent, (uint64_t)q.H * kMlaHeadRows, kMlaLatent * 2, 64, MN_W ? 64 : kFeat,
                    CU_TENSOR_MAP_SWIZZLE_128B) &&
        make_tma_3d(&x_map, bf, q.x, (uint64_t)q.K, (uint64_t)q.Hx, (uint64_t)q.R, (uint64_t)q.x_ld_h * 2,
                    (uint64_t)q.x_ld_r * 2, kStep, 1, N, CU_TENSOR_MAP_SWIZZLE_128B) &&
        make_tma_3d(&out_map, bf, q.out, (uint64_t)q.F, (uint64_t)q.Hx, (uint64_t)q.R, (uint64_t)q.F * 2,
                    (uint64_t)q.F * q.Hx * 2, 64, 1, chunk_of(N), CU_TENSOR_MAP_SWIZZLE_128B);
    if (!mapped) return NSA_ERR_CUDA;
    PParams p;
    p.ft_per_head = q.F / kFeat;
    p.n_ft = q.Hx * p.ft_per_head;
    p.n_rt = (int)ceil_div(q.R, N);
    p.steps = q.K / kStep;
    p.w_head_rows = q.w_head_rows;
    p.w_row0 = q.w_row0;
    p.status = q.status;
    const int64_t tiles = (int64_t)p.n_ft * p.n_rt;
    if (tiles > (1 << 30)) return NSA_ERR_UNSUPPORTED;
    NSA_CUDA_TRY(max_dynamic_smem<kern>(smem_of(N)));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles < sms ? tiles : sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_of(N);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    NSA_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, w_map, x_map, out_map, p));
    return NSA_OK;
}

nsa_status launch_pairs(const Problem &q, int sms, cudaStream_t stream)
{
    CUtensorMap w_map, x_map, out_map;
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const bool mapped =
        make_tma_2d(&w_map, bf, q.w, kMlaLatent, (uint64_t)q.H * kMlaHeadRows, kMlaLatent * 2, 64, kFeat, CU_TENSOR_MAP_SWIZZLE_128B) &&
        make_tma_3d(&x_map, bf, q.x, (uint64_t)q.K, 1, (uint64_t)q.R, (uint64_t)q.x_ld_h * 2, (uint64_t)q.x_ld_r * 2, kStep, 1,
                    kPairRows / 2, CU_TENSOR_MAP_SWIZZLE_128B) &&
        make_tma_3d(&out_map, bf, q.out, (uint64_t)q.F, 1, (uint64_t)q.R, (uint64_t)q.F * 2, (uint64_t)q.F * 2, 64, 1,
                    chunk_of(kPairRows), CU_TENSOR_MAP_SWIZZLE_128B);
    if (!mapped) return NSA_ERR_CUDA;
    PParams p = {};
    p.n_ft = q.F / (2 * kFeat);
    p.n_rt = (int)ceil_div(q.R, kPairRows);
    p.steps = q.K / kStep;
    p.status = q.status;
    const int64_t tiles = (int64_t)p.n_ft * p.n_rt;
    if (tiles > (1 << 30)) return NSA_ERR_UNSUPPORTED;
    NSA_CUDA_TRY(max_dynamic_smem<pair_product_kernel>(kPairSmem));
    const int pairs = sms / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = kPairSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    NSA_CUDA_TRY(cudaLaunchKernelEx(&cfg, pair_product_kernel, w_map, x_map, out_map, p));
    return NSA_OK;
}

// Whether nsa_mla_expand_kv's product goes to pairs: from three rounds of their tiles on.
bool pairs_for(const Problem &q, int sms)
{
    return q.all_heads && sms >= 2 && (int64_t)(q.F / (2 * kFeat)) * ceil_div(q.R, kPairRows) >= 3 * (sms / 2);
}

template <bool MN_W>
nsa_status launch_n(const Problem &q, cudaStream_t stream)
{
    const int sms = current_sm_count();
    if (sms <= 0) return NSA_ERR_CUDA;
    if (pairs_for(q, sms)) return launch_pairs(q, sms, stream);
    switch (pick_n(q, sms)) {
    case 16: return launch<16, MN_W>(q, sms, stream);
    case 32: return launch<32, MN_W>(q, sms, stream);
    case 64: return launch<64, MN_W>(q, sms, stream);
    case 128: return launch<128, MN_W>(q, sms, stream);
    default: return launch<256, MN_W>(q, sms, stream);
    }
}

// ---------------------------------------------------------------- rows of the cache

constexpr int kFp8Row = kMlaLatent + 16 + 2 * kMlaRope;
constexpr int kBf16Row = 2 * (kMlaLatent + kMlaRope);

__device__ __forceinline__ uint32_t dequantize2(uint32_t codes, float scale)
{
    const float lo = e4m3_to_float((uint8_t)(codes & 0xff)), hi = e4m3_to_float((uint8_t)(codes >> 8 & 0xff));
    return pack_bf16(__fmul_rn(lo, scale), __fmul_rn(hi, scale));
}

// A warp a row: the latent as bf16 into the workspace, the rope values into k_rope.
template <bool FP8>
__global__ void __launch_bounds__(256)
gather_rows_kernel(const uint8_t *kv, int64_t num_slots, const int32_t *slots, int m, uint8_t *latent, uint8_t *k_rope,
                   int32_t *status)
{
    pdl_trigger();  // the products' launch waits for this grid's end before it reads `latent`
    pdl_wait();
    const int i = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
    if (i >= m) return;
    const int64_t slot = slots[i];
    const bool there = slot >= 0 && slot < num_slots;
    if (slot >= num_slots && lane == 0) set_status(status, NSA_ERR_BOUNDS);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 a = zero, b = zero, r = zero;
    if (there) {
        const uint8_t *row = kv + slot * (FP8 ? kFp8Row : kBf16Row);
        if (FP8) {
            const uint4 w = *(const uint4 *)(row + 16 * lane);
            const float sc = *(const float *)(row + kMlaLatent + 4 * (lane / 8));
            a = make_uint4(dequantize2(w.x, sc), dequantize2(w.x >> 16, sc), dequantize2(w.y, sc), dequantize2(w.y >> 16, sc));
            b = make_uint4(dequantize2(w.z, sc), dequantize2(w.z >> 16, sc), dequantize2(w.w, sc), dequantize2(w.w >> 16, sc));
        } else {
            a = *(const uint4 *)(row + 32 * lane);
            b = *(const uint4 *)(row + 32 * lane + 16);
        }
        if (lane < 8) r = *(const uint4 *)(row + (FP8 ? kMlaLatent + 16 : 2 * kMlaLatent) + 16 * lane);
    }
    uint4 *o = (uint4 *)(latent + (int64_t)i * (2 * kMlaLatent) + 32 * lane);
    o[0] = a;
    o[1] = b;
    if (lane < 8) *(uint4 *)(k_rope + (int64_t)i * (2 * kMlaRope) + 16 * lane) = r;
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// Head h of row r at r * ld_r + h * ld_h: rows and heads that TMA can step over.
nsa_status check_strides(const void *x, int64_t ld_r, int64_t ld_h, int R, int H, int d)
{
    if ((H > 1 && ld_h < d) || (R > 1 && ld_r < d)) return NSA_ERR_INVALID_ARG;
    if (!aligned16(x) || (H > 1 && ld_h % 8) || (R > 1 && ld_r % 8)) return NSA_ERR_INVALID_ARG;
    if ((R > 1 && ld_r >= ((int64_t)1 << 38)) || (H > 1 && ld_h >= ((int64_t)1 << 38))) return NSA_ERR_UNSUPPORTED;
    return NSA_OK;
}

nsa_status head_product(const void *x_dev, int64_t ld_r, int64_t ld_h, const void *w_dev, int R, int H, int K, int F,
                        int w_row0, bool mn_w, void *out_dev, int32_t *status_dev, nsa_stream_t stream)
{
    if (R < 0 || H < 1) return NSA_ERR_INVALID_ARG;
    if (H > 65535 || R > (1 << 30)) return NSA_ERR_UNSUPPORTED;
    if (R == 0) return NSA_OK;
    if (!x_dev || !w_dev || !out_dev || !aligned16(w_dev) || !aligned16(out_dev) || ((uintptr_t)status_dev & 3))
        return NSA_ERR_INVALID_ARG;
    const nsa_status ok = check_strides(x_dev, ld_r, ld_h, R, H, K);
    if (ok != NSA_OK) return ok;
    // a single head's or row's stride is arbitrary
    if (H == 1) ld_h = K;
    if (R == 1) ld_r = ld_h * H;
    const Problem q = {w_dev, x_dev, ld_r, ld_h, out_dev, H, H, R, K, F, kMlaHeadRows, w_row0, mn_w, false, status_dev};
    return mn_w ? launch_n<true>(q, (cudaStream_t)stream) : launch_n<false>(q, (cudaStream_t)stream);
}

}  // namespace
}  // namespace nsa

extern "C" size_t nsa_mla_expand_kv_workspace_bytes(int m)
{
    return m > 0 ? (size_t)m * (2 * nsa::kMlaLatent) : 0;
}

extern "C" nsa_status nsa_mla_expand_kv(nsa_dtype kv_dtype, const void *kv_dev, int64_t num_slots, const int32_t *slots_dev,
                                        int m, const void *w_dev, int H, int d_latent, int d_rope, int d_nope, int d_v,
                                        void *kv_out_dev, void *k_rope_out_dev, void *workspace_dev,
                                        size_t workspace_bytes, int32_t *status_dev, nsa_stream_t stream)
{
    using namespace nsa;
    if (m < 0 || H < 1 || num_slots < 0) return NSA_ERR_INVALID_ARG;
    if ((kv_dtype != NSA_DT_BF16 && kv_dtype != NSA_DT_E4M3) || d_latent != kMlaLatent || d_rope != kMlaRope ||
        d_nope != kMlaNope || d_v != kMlaV || H > 65535 || m > (1 << 30))
        return NSA_ERR_UNSUPPORTED;
    if (m == 0) return NSA_OK;
    if (!kv_dev || !slots_dev || !w_dev || !kv_out_dev || !k_rope_out_dev || !workspace_dev || num_slots < 1)
        return NSA_ERR_INVALID_ARG;
    if (!aligned16(kv_dev) || !aligned16(w_dev) || !aligned16(kv_out_dev) || !aligned16(k_rope_out_dev) ||
        !aligned16(workspace_dev) || (((uintptr_t)slots_dev | (uintptr_t)status_dev) & 3) ||
        workspace_bytes < nsa_mla_expand_kv_workspace_bytes(m))
        return NSA_ERR_INVALID_ARG;
    const cudaStream_t s = (cudaStream_t)stream;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ceil_div(m, 8));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    NSA_CUDA_TRY(cudaLaunchKernelEx(&cfg, kv_dtype == NSA_DT_E4M3 ? gather_rows_kernel<true> : gather_rows_kernel<false>,
                                    (const uint8_t *)kv_dev, num_slots, slots_dev, m, (uint8_t *)workspace_dev,
                                    (uint8_t *)k_rope_out_dev, status_dev));
    // all heads' 256 features are one row of H * 256 values
    const Problem q = {w_dev, workspace_dev, kMlaLatent, kMlaLatent, kv_out_dev, H, 1, m, kMlaLatent, H * kMlaHeadRows,
                       0, 0, false, true, status_dev};
    return launch_n<false>(q, s);
}

extern "C" nsa_status nsa_mla_absorb_q(const void *q_nope_dev, int64_t nope_ld_r, int64_t nope_ld_h, const void *w_dev, int R,
                                       int H, int d_nope, int d_v, int d_latent, void *out_dev, int32_t *status_dev,
                                       nsa_stream_t stream)
{
    using namespace nsa;
    if (d_latent != kMlaLatent || d_nope != kMlaNope || d_v != kMlaV) return NSA_ERR_UNSUPPORTED;
    return head_product(q_nope_dev, nope_ld_r, nope_ld_h, w_dev, R, H, kMlaNope, kMlaLatent, 0, true, out_dev, status_dev,
                        stream);
}

extern "C" nsa_status nsa_mla_project_v(const void *latent_dev, int64_t latent_ld_r, int64_t latent_ld_h, const void *w_dev,
                                        int R, int H, int d_nope, int d_v, int d_latent, void *out_dev, int32_t *status_dev,
                                        nsa_stream_t stream)
{
    using namespace nsa;
    if (d_latent != kMlaLatent || d_nope != kMlaNope || d_v != kMlaV) return NSA_ERR_UNSUPPORTED;
    return head_product(latent_dev, latent_ld_r, latent_ld_h, w_dev, R, H, kMlaLatent, kMlaV, kMlaNope, false, out_dev,
                        status_dev, stream);
}
