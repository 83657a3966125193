// Tensor-core kernel of nsa_paged_mla for the 512 + 64 latent cache.
//
// A column is one (row, head) of a request; a CTA owns NC (16, 32 or 64) columns.  Per tile
// of 128 positions, as the sparse kernel does for its gathered rows:
//   S^T[128 keys, NC cols] = K_tile . Q^T                       (tcgen05, bf16)
//   P^T = 2^(scale S^T - m), m a lazily refreshed running maximum per column
//   O^T[512, NC cols] += V^T . P^T, V the first eight blocks of the same tile
// with O^T and S^T in TMEM (256 + 64 columns).  The sums of the unrounded P stay in
// fp32 registers (each thread its key's part) and are joined once at the end, so
// lse is good to fp32; P itself is rounded to bf16 for the product with V, whose
// operands must have one type (each weight off by at most 2^-8 of itself).
//
// Shared memory holds Q (72 KB of 64 columns) and one tile (144 KB), so tiles are pipelined
// by block pairs: pair m is loaded again as soon as O^T's d-block m, its last reader,
// is done, and S^T of the next tile starts on the pairs that have landed.  P^T lies
// in the rope block, which S^T has finished with.
//
// fp8 rows become bf16 in the CTA.  Up to 32 columns, Q leaves room for slots of raw codes,
// which TMA fills and 512 threads expand into the tile.  More columns leave none, and sharing
// the expansion pays: CTAs with neighbouring columns of the same request run as a cluster of two
// or four (make_plan), 128 threads of each expand their part of the tile from registers into a
// scratch in global memory that stays in L2, and every CTA of the cluster loads the tile from there.
//
// Every load goes into the CTA that issues it.  One load into all CTAs of a cluster took less
// from L2 (32 x 128 heads bf16 157 us, now 163; fp8 248, now 263; 8 x 4 x 128 heads fp8 704, now 683),
// but it is safe only on this GPU's own memory and in programs on one GPU, which a call cannot see.
//
// The tiles of all requests are cut into equal shares over the CTAs (teams of up to
// eight CTAs take the same tiles for different columns, so that a tile is read from
// HBM once).  A share that covers a request's columns only in part leaves raw sums,
// maxima and fp32 accumulators in the workspace, which paged_mla_join_kernel joins.
//
// Measured (GB300, a pass among others, positions 4096 .. 32768 unless said):
//   32 requests x 128 heads, bf16   163 us: 3.3 TB/s, 0.79 PF
//   128 x 16 heads, fp8, 1024 .. 16384    150 us: 3.2 TB/s
//   8 x 4 tokens x 128 heads, fp8, 16384 .. 131072   683 us: 0.78 PF
//   1 x 16 heads, bf16, 501         24 us, the host's part of a call; 12 us in a graph
// Bound by the chain of a tile: 5400 cycles (bf16, 64 columns), of which the products take 3640
// (N = 64 is bound by the tensor core's reads of shared memory: 48 cycles a product, not 32),
// the softmax 900 and the next tile's load behind its last reader the rest.  fp8 rows of up to 32
// columns: 6500 cycles, in which the threads that expand wait for the products of the one tile
// that shared memory holds.  17 thousand cycles pass before the first product.
#include <cstddef>

#include "paged_mla_tc.cuh"
#include "paged_tc.cuh"

namespace nsa {
namespace {

using namespace sm100;

constexpr int kCols = 64;                 // columns per CTA at most
constexpr uint32_t kKvBytes = 9 * kPtBlk;
constexpr uint32_t kColS = 256;           // S^T behind O^T's four blocks
constexpr uint32_t kTmemCols = 512;
constexpr float kRescale = 8.0f;          // log2 units
// The running maximum of a column that has seen no score yet: finite, so that a score of -inf gets the
// exponent -inf (weight 0) from it and not NaN, and so low that any other score asks for a new maximum.
constexpr float kNoMax = -3.402823466e38f;
constexpr int kMaxTeam = 8;
// How the tile's rows come: a bf16 cache by TMA; raw fp8 rows by TMA into slots beside the
// tile and expanded from there; or fp8 rows expanded into the CTA's scratch in global memory
// (each CTA of a cluster its part of the tile) and loaded from it in whole blocks.
enum Rows { kBf16Rows, kRawRows, kScratchRows };
// What a further request in a share costs, in tiles: its epilogue, the loads that find it and its
// first tiles from HBM took 18 - 22 thousand cycles against 5.2 a tile (32 requests of 128 heads:
// the last share ended at 163 us, the median at 145, when shares were cut by tiles alone; 2 and 3
// tiles instead of 4 were 4 % and 1 % slower).  fp8 tiles take longer, and their first ones do not.
constexpr int piece_of(Rows rows) { return rows == kBf16Rows ? 4 : 2; }
// Softmax groups of four warps, one key a thread and kGrp columns a group: 16 columns keep a
// thread's exponents and sums in 72 registers, which leaves room for the row warps.
constexpr int grp_of(int nc) { return nc == 16 ? 8 : 16; }
constexpr int row0_of(int nc) { return 128 + 128 * (nc / grp_of(nc)); }  // first row-expanding thread
constexpr int threads_of(Rows rows, int nc)
{
    return row0_of(nc) + (rows == kRawRows ? kDqThreads : rows == kScratchRows ? kScrThreads : 0);
}

struct AShared {
    alignas(16) float m_run[kCols];   // running maximum, log2 units
    alignas(16) float alpha[kCols];
    float red[4][kCols];
    float inv[kCols];                 // 1 / sum; 0: no key
    int len[kCols];                   // positions the column's row sees
    int min_len[4];                   // shortest of all the CTA's columns, one copy a group
    int odd0[4], odd1[4];             // first and last position of the piece whose row was made finite (one copy a group)
    uint64_t pair_full[5];            // block pair m of the tile landed (m = 4: the rope block)
    uint64_t pair_free[5];            // its readers are done (m = 4: every product of the tile)
    uint64_t q_full, q_empty, s_full, p_full, o_fin;
    RawShared raw;
    // tiles of the scratch: this CTA's part written (its row warps), every CTA's part written, the tile loaded into this CTA
    uint64_t scr_part[kScrMaxSlots], scr_full[kScrMaxSlots], scr_loaded[kScrMaxSlots];
    TileShare share;
    uint32_t tmem_base;
    volatile uint32_t scr_tiles;      // parts of tiles that the row warps have expanded
    volatile int abort;
};
constexpr int raw_slots(int nc) { return nc == 16 ? 3 : 2; }  // as many as fit beside Q and the tile
constexpr size_t smem_of(Rows rows, int nc)
{
    return 1024 + 9 * (size_t)nc * 128 + kKvBytes + (rows == kRawRows ? raw_slots(nc) * kRawSlot + 2 * kScaleSlot : 0) +
           sizeof(AShared);
}
static_assert(smem_of(kBf16Rows, 64) <= 232448 && smem_of(kRawRows, 32) <= 232448 && smem_of(kRawRows, 16) <= 232448,
              "shared memory per CTA");

struct AParams {
    PagedTc t;
    int cols, nc, groups, team, mult;  // columns per request and per CTA, groups of nc, CTAs per team, groups / team
    int teams;
    int slot_cols;                 // columns of a partial slot
    __nv_bfloat16 *out;
    float *lse;
    int4 *unit;                    // [B * mult] of each (request, group set): first and last share, whether the first began earlier
    float *part;                   // [2 * CTAs][slot_cols][512] raw accumulators
    float2 *part_ml;               // [2 * CTAs][slot_cols] maximum (log2 units) and sum
    uint8_t *scratch;              // [clusters][scr_slots] tiles of bf16 (fp8 rows of clusters)
};

// The pieces of a share: tiles [t0, t1) of group set j of request b.
struct Seg {
    int b, j, t0, t1, len;
    int left;  // places of the share behind this piece

    __device__ __forceinline__ bool start(const AParams &p, const TileShare &s)
    {
        left = (int)(s.g1 - s.g0);
        if (left <= 0) return false;
        b = s.b;
        len = s.len;
        const int places = tiles_of(len) + s.piece;
        j = s.off < 0x100000000LL ? (int)((uint32_t)s.off / (uint32_t)places) : (int)(s.off / places);
        return enter((int)(s.off - (int64_t)j * places), s.piece);
    }
    // the unit from place `at` on; false if the share ends before its next tile
    __device__ __forceinline__ bool enter(int at, int piece)
    {
        const int end = min(tiles_of(len) + piece, at + left);
        left -= end - at;
        t0 = max(0, at - piece);
        t1 = max(0, end - piece);
        return t1 > t0;
    }
    __device__ __forceinline__ bool next(const AParams &p, const TileShare &s)
    {
        if (left <= 0) return false;
        if (++j == p.mult) {
            j = 0;
            do {
                if (++b >= p.t.B) return false;
                len = request_len(p.t, b);
            } while (len == 0);
        }
        return enter(0, s.piece);
    }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles_of(len); }
};
constexpr int64_t kMaxShare = 1 << 30;  // places of a share, so that a place and `left` stay ints

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ bool not_finite(uint32_t f32) { return (f32 & 0x7f800000u) == 0x7f800000u; }
// Two bf16 with what is not finite replaced by 0.
__device__ __forceinline__ uint32_t finite_pair(uint32_t w)
{
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
    if ((w & 0x00007f80u) == 0x00007f80u) w &= 0xffff0000u;
    return w;
}

// A column's values of all lanes joined, by halving exchanges: lane x gets that of column x % G.
template <int G, class Join>
__device__ __forceinline__ float over_lanes(float (&v)[G], int lane, Join join)
{
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int c = 0; c < o; ++c) {
            const float give = up ? v[c] : v[c + o];
            const float got = __shfl_xor_sync(0xffffffffu, give, o);
            v[c] = join(up ? v[c + o] : v[c], got);
        }
    }
#pragma unroll
    for (int o = G; o < 32; o <<= 1) v[0] = join(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    return v[0];
}

// G columns of the accumulator at `taddr` from or into TMEM, one lane a thread.
template <int G>
__device__ __forceinline__ void tmem_ldg(uint32_t taddr, uint32_t (&r)[G])
{
    if constexpr (G == 32) tmem_ld32(taddr, r);
    else if constexpr (G == 16) tmem_ld16(taddr, r);
    else tmem_ld8(taddr, r);
    tmem_ld_wait();
}
template <int G>
__device__ __forceinline__ void tmem_stg(uint32_t taddr, const uint32_t (&r)[G])
{
    if constexpr (G == 32) tmem_st32(taddr, r);
    else if constexpr (G == 16) tmem_st16(taddr, r);
    else tmem_st8(taddr, r);
}

// Which columns of a group (`len`: what they see) see a value that is not finite among components d, d + 128,
// d + 256 and d + 384 of positions pos0 .. pos1: bit 16 m + c for component d + 128 m and column c.  Not
// inlined: it is rarely called, and its registers would be taken from the tile loop.
template <int KDT, int G>
__device__ __noinline__ uint64_t hidden_values(const uint8_t *kv, int64_t num_pages, int ps, const int32_t *pt, int pos0,
                                               int pos1, const int *len, int d)
{
    uint64_t bits = 0;
#pragma unroll 1
    for (int pos = pos0; pos <= pos1; ++pos) {
        const int page = __ldg(pt + pos / ps);
        if (page < 0 || page >= num_pages) continue;
        const int64_t slot = (int64_t)page * ps + pos % ps;
        uint32_t see = 0;
        for (int c = 0; c < G; ++c) see |= (pos < len[c] ? 1u : 0u) << c;
#pragma unroll
        for (int m = 0; m < 4; ++m)
            if (not_finite(__float_as_uint(load_cache<KDT>(kv, slot, m * 128 + d, kPtDl, kPtDr))))
                bits |= (uint64_t)see << (16 * m);
    }
    return bits;
}

// CL: CTAs of a cluster, which share the expansion of their tiles; NC: columns of the CTA's products (16, 32 or 64).
// kv_map: bf16 rows of the cache, or the fp8 codes; sc_map, rope_map: of raw rows.  Scratch rows need none.
template <Rows ROWS, int CL, int NC>
__global__ void __launch_bounds__(threads_of(ROWS, NC), 1)
paged_mla_tc_kernel(AParams p, const __grid_constant__ CUtensorMap qn_map, const __grid_constant__ CUtensorMap qr_map,
                    const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap sc_map,
                    const __grid_constant__ CUtensorMap rope_map)
{
    constexpr bool RAW = ROWS == kRawRows, SCR = ROWS == kScratchRows;
    constexpr int kScrRows = kPtTok / CL;     // rows of a tile that one CTA expands
    constexpr int kScrAhead = scr_ahead(CL), kScrSlots = scr_slots(CL);
    constexpr int kGrp = grp_of(NC), kGroups = NC / kGrp, kRow0 = row0_of(NC), kRaw = raw_slots(NC);
    constexpr uint32_t kQBlk = NC * 128;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *q_s = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *kv_s = q_s + (9 * kQBlk + 1023) / 1024 * 1024;
    uint8_t *p_s = kv_s + 8 * kPtBlk;  // P^T in the rope block
    uint8_t *raw_s = kv_s + kKvBytes, *sc_s = raw_s + (RAW ? kRaw * kRawSlot : 0);
    AShared *sm = (AShared *)(sc_s + (RAW ? 2 * kScaleSlot : 0));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int team = blockIdx.x / p.team, rank = blockIdx.x - team * p.team;  // rank: column group in the set
    const int peer = CL > 1 ? (int)cluster_ctarank() : 0;
    uint8_t *scr = SCR ? p.scratch + (int64_t)(blockIdx.x / CL) * kScrSlots * kScrTile : nullptr;  // of the cluster

    if (threadIdx.x == 0) {
        for (int m = 0; m < 5; ++m) {
            mbar_init(&sm->pair_full[m], RAW && m < 4 ? kDqThreads / 32 : 1);
            mbar_init(&sm->pair_free[m], 1);
        }
        mbar_init(&sm->q_full, 1);
        mbar_init(&sm->q_empty, 1);
        mbar_init(&sm->s_full, 1);
        mbar_init(&sm->p_full, 128 * kGroups);
        mbar_init(&sm->o_fin, 1);
        for (int i = 0; i < kMaxRaw; ++i) {
            mbar_init(&sm->raw.full[i], 1);
            mbar_init(&sm->raw.empty[i], kDqThreads / 32);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&sm->raw.tile_full[i], 1);
        for (int i = 0; i < kScrMaxSlots; ++i) {
            mbar_init(&sm->scr_part[i], kScrThreads / 32);
            mbar_init(&sm->scr_full[i], CL);
            mbar_init(&sm->scr_loaded[i], 1);
        }
        sm->scr_tiles = 0;
        sm->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&sm->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    if (threadIdx.x == 64) {
        prefetch_tensormap(&qn_map);
        prefetch_tensormap(&qr_map);
        if (!SCR) prefetch_tensormap(&kv_map);
    }
    pdl_trigger();  // the join may be launched while this grid works; it waits for its end
    tc_fence_before();
    find_share(p.t, p.mult, piece_of(ROWS), team, p.teams, &sm->share);  // ends with a block barrier
    if (CL > 1) cluster_sync_all();  // the peers' barriers are ready before anything reaches them
    tc_fence_after();
    const uint32_t tmem = sm->tmem_base;
    auto fail = [&]() {
        sm->abort = 1;
        set_status(p.t.status, NSA_ERR_TIMEOUT);
    };
    // The shares of every unit, for the join (one warp of the launch).
    auto write_units = [&]() {
        const int64_t total = sm->share.total, np = sm->share.np;
        const int piece = sm->share.piece;
        // share k is [total * k / np, total * (k + 1) / np)
        auto share_of = [&](int64_t g) -> int {
            int k = (int)(g * np / total);
            while (k + 1 < np && total * (k + 1) / np <= g) ++k;
            while (k > 0 && total * k / np > g) --k;
            return k;
        };
        int64_t before = 0;
        for (int base = 0; base < p.t.B; base += 32) {
            const int b = base + lane;
            const int tiles = b < p.t.B ? tiles_of(request_len(p.t, b)) : 0;
            const int64_t v = tiles > 0 ? tiles + piece : 0;
            int64_t inc = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += x;
            }
            if (b < p.t.B) {
                int64_t u0 = (before + inc - v) * p.mult;
                for (int j = 0; j < p.mult; ++j, u0 += v) {
                    int4 u = make_int4(0, 0, 0, 0);
                    if (v > 0) {
                        u.x = share_of(u0 + piece);
                        u.y = share_of(u0 + v - 1);
                        u.z = total * u.x / np < u0 ? 1 : 0;
                    }
                    p.unit[(int64_t)b * p.mult + j] = u;
                }
            }
            before += __shfl_sync(0xffffffffu, inc, 31);
        }
    };
    Seg s;
    const bool work = s.start(p, sm->share);

    if (warp < 4) {
        if (warp == 0 && work) {
            // -------------------------------------------------------- TMA
            const int boxes = kPtTok / p.t.box_rows;  // at most 16, one a lane
            const uint32_t box_bytes = (uint32_t)p.t.box_rows * 128;
            constexpr uint32_t kRowBytes = ROWS == kBf16Rows ? 2 * (kPtDl + kPtDr) : kPtFp8Row;
            uint32_t i = 0, seg = 0, rph = 0;
            int rs = 0;
            bool ok = true;
            for (bool more = true; more && ok; more = s.next(p, sm->share), ++seg) {
                if (seg > 0 && !mbar_wait(&sm->q_empty, (seg - 1) & 1, kPtWait)) ok = false;
                const int row = s.b * p.cols + (s.j * p.team + rank) * NC;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&sm->q_full, 9 * kQBlk);
                    for (int c = 0; c < 8; ++c) tma_load_2d(q_s + c * kQBlk, &qn_map, 64 * c, row, &sm->q_full);
                    tma_load_2d(q_s + 8 * kQBlk, &qr_map, 0, row, &sm->q_full);
                }
                __syncwarp();
                const int32_t *pt = p.t.page_table + (int64_t)s.b * p.t.pt_ld;
                // row of this lane's box of tile t, or -1
                auto box_row = [&](int t) -> int {
                    const int pos = t * kPtTok + lane * p.t.box_rows;
                    const int page = lane < boxes && t < s.t1 ? checked_page(p.t, pt, pos, s.len) : -1;
                    return page < 0 ? -1 : page * p.t.ps + pos % p.t.ps;
                };
                int y = box_row(s.t0), y1 = box_row(s.t0 + 1);
                for (int t = s.t0; t < s.t1 && ok; ++t, ++i) {
                    const uint32_t live = __ballot_sync(0xffffffffu, y >= 0);
                    const uint32_t blk_bytes = SCR ? kPtBlk : __popc(live) * box_bytes;
                    // one lane issues a box at a time from uniform registers: a box's coordinates and
                    // addresses per lane took 350 cycles a pair
                    const int y_first = __shfl_sync(0xffffffffu, y, 0);
                    auto boxes_of = [&](auto issue) {
                        int yb = y_first;
                        for (int x = 0; x < boxes; ++x) {
                            if (x > 0) yb = __shfl_sync(0xffffffffu, y, x);
                            if (yb >= 0 && elect_one()) issue(x, yb);
                            __syncwarp();
                        }
                    };
                    if constexpr (RAW) {
#pragma unroll 1
                        for (int m = 0; m < 4; ++m) {
                            if (!mbar_wait(&sm->raw.empty[rs], rph ^ 1, kPtWait)) ok = false;
                            if (elect_one()) {
                                if (m == 0) {
                                    sm->raw.boxes[i & 1] = live;
                                    mbar_arrive_expect_tx(&sm->raw.tile_full[i & 1], blk_bytes / 8);
                                }
                                mbar_arrive_expect_tx(&sm->raw.full[rs], blk_bytes);
                            }
                            __syncwarp();
                            boxes_of([&](int x, int yb) {
                                tma_load_2d(raw_s + rs * kRawSlot + x * box_bytes, &kv_map, 128 * m, yb, &sm->raw.full[rs]);
                                if (m == 0)
                                    tma_load_2d(sc_s + (i & 1) * kScaleSlot + x * (box_bytes / 8), &sc_map, kPtDl, yb,
                                                &sm->raw.tile_full[i & 1]);
                            });
                            if (++rs == kRaw) {
                                rs = 0;
                                rph ^= 1;
                            }
                        }
                        if (!mbar_wait(&sm->pair_free[4], (i & 1) ^ 1, kPtWait)) ok = false;
                        if (elect_one()) mbar_arrive_expect_tx(&sm->pair_full[4], blk_bytes);
                        __syncwarp();
                        boxes_of([&](int x, int yb) {
                            tma_load_2d(kv_s + 8 * kPtBlk + x * box_bytes, &rope_map, kFp8RopeX, yb, &sm->pair_full[4]);
                        });
                    } else {
                        const uint32_t ss = i % kScrSlots;
                        if constexpr (SCR) {
                            // every CTA's row warps have written their part of the tile to its scratch
                            if (!mbar_wait_cluster(&sm->scr_full[ss], i / kScrSlots & 1, kPtWait)) ok = false;
                            asm volatile("fence.proxy.async.global;" ::: "memory");
                        }
#pragma unroll
                        for (int m = 0; m < 5; ++m) {
                            if (!mbar_wait(&sm->pair_free[m], (i & 1) ^ 1, kPtWait)) ok = false;
                            if (elect_one()) {
                                mbar_arrive_expect_tx(&sm->pair_full[m], (m < 4 ? 2 : 1) * blk_bytes);
                                if (SCR && CL == 4 && m == 4 && i > 0) mbar_arrive(&sm->scr_loaded[(i - 1) % kScrSlots]);
                            }
                            __syncwarp();
                            if constexpr (SCR) {
                                if (elect_one())
                                    bulk_load(kv_s + 2 * m * kPtBlk, scr + ss * kScrTile + 2 * m * kPtBlk,
                                              (m < 4 ? 2 : 1) * kPtBlk, &sm->pair_full[m]);
                                __syncwarp();
                            } else {
                                boxes_of([&](int x, int yb) {
#pragma unroll
                                    for (int c = 2 * m; c < (m < 4 ? 2 * m + 2 : 9); ++c)
                                        tma_load_2d(kv_s + c * kPtBlk + x * box_bytes, &kv_map, 64 * c, yb, &sm->pair_full[m]);
                                });
                            }
                        }
                    }
                    // the tile after the next one into L2 while this one is worked on
                    const int y2 = SCR ? -1 : box_row(t + 2);
                    if (!SCR && y2 >= 0)
                        prefetch_l2_bulk(p.t.kv + (int64_t)y2 * kRowBytes, (uint32_t)p.t.box_rows * kRowBytes);
                    y = y1;
                    y1 = y2;
                    ok = __all_sync(0xffffffffu, ok && !sm->abort) != 0;
                }
                ok = __all_sync(0xffffffffu, ok && !sm->abort) != 0;
            }
            if (!ok && lane == 0) fail();
            if (lane == 0) {  // nothing is in flight at the end
                if (i > 0)
                    for (int m = 0; m < 5; ++m) {
                        mbar_wait(&sm->pair_full[m], (i - 1) & 1, kPtWait);
                        mbar_wait(&sm->pair_free[m], (i - 1) & 1, kPtWait);
                    }
                if (RAW) {
                    for (uint32_t x = i > 2 ? i - 2 : 0; x < i; ++x) mbar_wait(&sm->raw.tile_full[x & 1], (x >> 1) & 1, kPtWait);
                    for (int x = 0; x < kRaw; ++x) mbar_wait(&sm->raw.full[x], x < rs ? rph : rph ^ 1, kPtWait);
                }
                if (seg > 0) mbar_wait(&sm->q_full, (seg - 1) & 1, kPtWait);
            }
            __syncwarp();
        } else if (warp == 1 && work) {
            // -------------------------------------------------------- MMA
            // The whole warp walks and waits; one lane issues, with descriptors in uniform registers
            // (a lane-0 branch around the loop took 90 - 110 cycles an instruction).
            const uint32_t idesc_s = instr_desc(1, 1, 0, 0, kPtTok, NC);  // K-major A and B
            const uint32_t idesc_o = instr_desc(1, 1, 1, 1, 128, NC);     // MN-major A and B
            const uint64_t k_desc = smem_desc(smem_u32(kv_s), 16, 1024, kSwizzle128B);
            const uint64_t q_desc = smem_desc(smem_u32(q_s), 16, 1024, kSwizzle128B);
            const uint64_t v_desc = smem_desc(smem_u32(kv_s), kPtBlk, 1024, kSwizzle128B);
            const uint64_t p_desc = smem_desc(smem_u32(p_s), kPtBlk, 1024, kSwizzle128B);
            uint32_t i = 0, seg = 0;
            bool ok = true;
            for (bool more = true; more && ok; more = s.next(p, sm->share), ++seg) {
                if (!mbar_wait(&sm->q_full, seg & 1, kPtWait)) ok = false;
                for (int t = s.t0; t < s.t1 && ok; ++t, ++i) {
#pragma unroll
                    for (int m = 0; m < 5; ++m) {
                        if (!mbar_wait(&sm->pair_full[m], i & 1, kPtWait)) ok = false;
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int c = 2 * m; c < (m < 4 ? 2 * m + 2 : 9); ++c)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mma_f16(tmem + kColS, k_desc + (c * kPtBlk + k * 32) / 16,
                                            q_desc + (c * kQBlk + k * 32) / 16, idesc_s, (c | k) != 0);
                            if (m == 4) {
                                mma_commit(&sm->s_full);
                                if (t + 1 == s.t1) mma_commit(&sm->q_empty);
                            }
                        }
                        __syncwarp();
                    }
                    if (!mbar_wait(&sm->p_full, i & 1, kPtWait)) ok = false;
                    ok = __all_sync(0xffffffffu, ok && !sm->abort) != 0;
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
#pragma unroll
                            for (int k = 0; k < kPtTok / 16; ++k)
                                mma_f16(tmem + m * NC, v_desc + (2 * m * kPtBlk + k * 2048) / 16, p_desc + k * 2048 / 16,
                                        idesc_o, k > 0 ? 1u : (uint32_t)(t > s.t0));
                            mma_commit(&sm->pair_free[m]);
                        }
                        mma_commit(&sm->pair_free[4]);
                        if (t + 1 == s.t1) mma_commit(&sm->o_fin);
                    }
                    __syncwarp();
                }
                ok = __all_sync(0xffffffffu, ok && !sm->abort) != 0;
            }
            if (!ok) {
                if (lane == 0) fail();
                // whatever was issued is done before shared memory and TMEM are given up
                if (elect_one()) mma_commit(&sm->o_fin);
                __syncwarp();
                for (int w = 0; w < 2; ++w) mbar_wait(&sm->o_fin, w, kPtWait / 100);
            }
            __syncwarp();
        } else if (warp == 2) {
            if constexpr (SCR) {
                // ---------------------------------------------------- tells the cluster of this CTA's parts of tiles
                // A warp of its own: a release to other CTAs waits until the row warps' stores have arrived, a
                // thousand cycles and more, which they need not spend (279 us for 32 x 128 heads when they did).
                uint32_t i = 0;
                bool ok = true;
                for (bool more = work; more && ok; more = s.next(p, sm->share))
                    for (int t = s.t0; t < s.t1 && ok; ++t, ++i) {
                        const uint32_t ss = i % kScrSlots;
                        if (!mbar_wait(&sm->scr_part[ss], i / kScrSlots & 1, kPtWait)) ok = false;
                        if (lane < CL) mbar_arrive_cluster(&sm->scr_full[ss], lane);
                        ok = __all_sync(0xffffffffu, ok && !sm->abort) != 0;
                    }
                if (!ok && lane == 0) fail();
            } else if (blockIdx.x == 0) {
                write_units();
            }
        } else if (warp == 3) {
            // -------------------------------------------------------- bad lengths, requests without a key
            if (SCR && blockIdx.x == 0) write_units();
            if (blockIdx.x == 0) report_lengths(p.t, lane, 32);
            for (int b = blockIdx.x; b < p.t.B; b += gridDim.x) {
                if (request_len(p.t, b) > 0) continue;
                const int64_t row0 = (int64_t)b * p.cols;
                uint4 *o = reinterpret_cast<uint4 *>(p.out + row0 * kPtDl);
                if (((uintptr_t)p.out & 15) == 0)
                    for (int64_t e = lane; e < (int64_t)p.cols * (kPtDl / 8); e += 32) o[e] = make_uint4(0u, 0u, 0u, 0u);
                else
                    for (int64_t e = lane; e < (int64_t)p.cols * kPtDl; e += 32) p.out[row0 * kPtDl + e] = __float2bfloat16_rn(0.f);
                for (int c = lane; c < p.cols; c += 32) p.lse[row0 + c] = -INFINITY;
            }
            if (SCR && work) {
                // ---------------------------------------------------- rows into L2 ahead of the row warps
                constexpr int kAhead = 3;
                constexpr int kPolls = 1 << 22;  // about a second
                const int per = kScrRows / p.t.box_rows;  // boxes of this CTA's part of a tile
                Seg f = s;
                int ft = f.t0;
                bool fetch = true;
                auto prefetch = [&](bool wanted) {
                    const int pos = ft * kPtTok + peer * kScrRows + lane * p.t.box_rows;
                    if (wanted && lane < per && pos < f.len) {
                        const int page = __ldg(p.t.page_table + (int64_t)f.b * p.t.pt_ld + pos / p.t.ps);
                        if (page >= 0 && page < p.t.num_pages)
                            prefetch_l2_bulk(p.t.kv + ((int64_t)page * p.t.ps + pos % p.t.ps) * kPtFp8Row,
                                             (uint32_t)p.t.box_rows * kPtFp8Row);
                    }
                    if (++ft >= f.t1) {
                        fetch = f.next(p, sm->share);
                        ft = f.t0;
                    }
                };
                // Paced by a count, not by the barriers' phases: the requests without a key may have
                // kept this warp busy for several tiles, which it then passes over.
                for (uint32_t n = 0; fetch; ++n) {
                    uint32_t done = sm->scr_tiles;
                    for (int x = 0; done + kAhead <= n && !sm->abort && x < kPolls; ++x) {
                        __nanosleep(200);
                        done = sm->scr_tiles;
                    }
                    if (done + kAhead <= n) break;
                    prefetch(n >= done);
                }
                __syncwarp();
            }
        }
    } else if (warp < 4 + 4 * kGroups) {
        if (work) {
            // -------------------------------------------------------- softmax: one key a thread, kGrp columns a group
            const int grp = (warp - 4) >> 2, quad = warp & 3, cb = grp * kGrp, bar = 1 + grp;
            const int key = quad * 32 + lane, et = (threadIdx.x - 128) & 127;
            const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
            const float4 *m4 = reinterpret_cast<const float4 *>(sm->m_run + cb);
            uint32_t i = 0, seg = 0;
            bool ok = true;
            for (bool more = true; more && ok; more = s.next(p, sm->share), ++seg) {
                const int col0 = (s.j * p.team + rank) * NC;  // first column of this CTA in the request
                if (et < 32) {
                    int shortest = 0x7fffffff;
                    for (int cc = lane; cc < NC; cc += 32) {
                        const int c = col0 + cc;
                        int len = 0x7fffffff;  // padding: never masked, never written
                        if (c < p.cols) {
                            const int L = p.t.row_len[(int64_t)s.b * p.t.n + c / p.t.H];
                            len = L >= 0 && L <= p.t.max_row_len ? L : 0;
                        }
                        shortest = min(shortest, len);
                        if (cc >= cb && cc < cb + kGrp) {
                            sm->len[cc] = len;
                            sm->m_run[cc] = kNoMax;
                        }
                    }
                    shortest = __reduce_min_sync(0xffffffffu, shortest);
                    if (lane == 0) {
                        sm->min_len[grp] = shortest;
                        sm->odd0[grp] = 0x7fffffff;
                        sm->odd1[grp] = -1;
                    }
                }
                bar_sync(bar, 128);
                const int min_len = sm->min_len[grp];
                const int32_t *pt = p.t.page_table + (int64_t)s.b * p.t.pt_ld;
                float2 l[kGrp / 2];
#pragma unroll
                for (int c = 0; c < kGrp / 2; ++c) l[c] = make_float2(0.f, 0.f);
                for (int t = s.t0; t < s.t1; ++t, ++i) {
                    const int pos = t * kPtTok + key;
                    const bool valid = checked_page(p.t, pt, pos, s.len) >= 0;
                    ok = mbar_wait(&sm->s_full, i & 1, kPtWait);
                    if (!ok) fail();
                    // S^T is done, so the tile was loaded (clusters of four: told by the TMA warp, later)
                    if (SCR && CL == 2 && threadIdx.x == 128 && ok) mbar_arrive(&sm->scr_loaded[i % kScrSlots]);
                    tc_fence_after();
                    const bool whole = (t + 1) * kPtTok <= min_len && __all_sync(0xffffffffu, valid);
                    bool odd = false;  // a score of this key is not finite (looked at where columns are masked)
                    // exponents d = x - m; a key above its column's maximum by 2^8 asks for new maxima
                    float2 d[kGrp / 2];
                    auto exponents = [&]() {
                        uint32_t sa[kGrp];
                        tmem_ldg<kGrp>(lanes + kColS + cb, sa);
                        const float2 sc = make_float2(p.t.scale_log2, p.t.scale_log2);
#pragma unroll
                        for (int c = 0; c < kGrp / 4; ++c) {
                            const float4 m = m4[c];
                            d[2 * c] = fma2(make_float2(__uint_as_float(sa[4 * c]), __uint_as_float(sa[4 * c + 1])), sc,
                                            make_float2(-m.x, -m.y));
                            d[2 * c + 1] = fma2(make_float2(__uint_as_float(sa[4 * c + 2]), __uint_as_float(sa[4 * c + 3])),
                                                sc, make_float2(-m.z, -m.w));
                        }
                        if (!whole) {
                            odd = not_finite(sa[0]);
#pragma unroll
                            for (int c = 0; c < kGrp / 2; ++c) {
                                if (!valid || pos >= sm->len[cb + 2 * c]) d[c].x = -INFINITY;
                                if (!valid || pos >= sm->len[cb + 2 * c + 1]) d[c].y = -INFINITY;
                            }
                        }
                    };
                    exponents();
                    float top = d[0].x;
#pragma unroll
                    for (int c = 0; c < kGrp / 2; ++c) top = fmaxf(fmaxf(top, d[c].x), d[c].y);
                    if (bar_red_or(bar, 128, !ok || sm->abort || top > kRescale)) {
                        if (bar_red_or(bar, 128, !ok || sm->abort)) { ok = false; break; }
                        // new maxima from this tile; sums and accumulators so far are rescaled
                        {
                            uint32_t sa[kGrp];
                            tmem_ldg<kGrp>(lanes + kColS + cb, sa);
                            float v[kGrp];
#pragma unroll
                            for (int c = 0; c < kGrp; ++c)
                                v[c] = valid && pos < sm->len[cb + c] ? __uint_as_float(sa[c]) * p.t.scale_log2 : -INFINITY;
                            const float top = over_lanes(v, lane, [](float x, float y) { return fmaxf(x, y); });
                            if (lane < kGrp) sm->red[quad][cb + lane] = top;
                        }
                        bar_sync(bar, 128);
                        if (et < kGrp) {
                            const int c = cb + et;
                            const float cm = fmaxf(fmaxf(sm->red[0][c], sm->red[1][c]), fmaxf(sm->red[2][c], sm->red[3][c]));
                            const float mo = sm->m_run[c], mn = fmaxf(mo, cm);
                            sm->alpha[c] = exp2f(mo - mn);
                            sm->m_run[c] = mn;
                        }
                        bar_sync(bar, 128);
                        if (t > s.t0) {
                            // S^T of this tile is done, and with it the products of the tile before
#pragma unroll 1
                            for (int m = 0; m < 4; ++m) {
                                uint32_t v[kGrp];
                                tmem_ldg<kGrp>(lanes + m * NC + cb, v);
#pragma unroll
                                for (int c = 0; c < kGrp; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * sm->alpha[cb + c]);
                                tmem_stg<kGrp>(lanes + m * NC + cb, v);
                            }
                            tmem_st_wait();
#pragma unroll
                            for (int c = 0; c < kGrp / 2; ++c) {
                                l[c].x *= sm->alpha[cb + 2 * c];
                                l[c].y *= sm->alpha[cb + 2 * c + 1];
                            }
                        }
                        exponents();
                    }
#pragma unroll
                    for (int c8 = 0; c8 < kGrp / 8; ++c8) {
                        uint32_t pk[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int c = 4 * c8 + k;
                            const float2 e = make_float2(ex2_approx(d[c].x), ex2_approx(d[c].y));
                            l[c] = add2(l[c], e);
                            pk[k] = pack2(e.x, e.y);
                        }
                        *reinterpret_cast<uint4 *>(p_s + sw128_offset(key, cb / 8 + c8)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
                    // A weight of 0 does not hide what is not finite, so it is taken out of this group's share
                    // of the key's latent blocks (S^T has read them): all of a row that is not there, and from
                    // a row that only some columns see the values that are not finite.  Such a value makes every
                    // column's score of the key not finite, which is how it is noticed.  The columns that see the
                    // key get NaN sums from a score of NaN or +inf; what 0 x inf gives those whose score is -inf
                    // is put back at the end of the piece.
                    const bool absent = ROWS == kBf16Rows && !valid;
                    if (absent || (odd && valid && pos >= min_len)) {
                        if (!absent) {
                            atomicMin(&sm->odd0[grp], pos);
                            atomicMax(&sm->odd1[grp], pos);
                        }
                        for (int m = 0; m < 4; ++m) mbar_wait(&sm->pair_full[m], i & 1, kPtWait);
#pragma unroll 1
                        for (int c = grp * (8 / kGroups); c < (grp + 1) * (8 / kGroups); ++c) {
                            uint4 *r = reinterpret_cast<uint4 *>(kv_s + c * kPtBlk + key * 128);
#pragma unroll 1
                            for (int k = 0; k < 8; ++k) {
                                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                                if (!absent) {
                                    v = r[k];
                                    v.x = finite_pair(v.x);
                                    v.y = finite_pair(v.y);
                                    v.z = finite_pair(v.z);
                                    v.w = finite_pair(v.w);
                                }
                                r[k] = v;
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    tc_fence_before();
                    mbar_arrive(&sm->p_full);
                }
                if (!ok) break;
                // ---------------------------------------------------- the piece's sums and accumulators
                float ls[kGrp];
#pragma unroll
                for (int c = 0; c < kGrp / 2; ++c) {
                    ls[2 * c] = l[c].x;
                    ls[2 * c + 1] = l[c].y;
                }
                const float part = over_lanes(ls, lane, [](float x, float y) { return x + y; });
                if (lane < kGrp) sm->red[quad][cb + lane] = part;
                bar_sync(bar, 128);
                const int odd0 = sm->odd0[grp], odd1 = sm->odd1[grp];
                const bool whole = s.whole();
                const int nc = min(kGrp, p.cols - col0 - cb);  // real columns of this group (may be <= 0)
                const int64_t row0 = (int64_t)s.b * p.cols + col0 + cb;
                const int64_t slot = (int64_t)blockIdx.x * 2 + (seg > 0 ? 1 : 0);
                if (et < kGrp) {
                    const int c = cb + et;
                    const float sum = (sm->red[0][c] + sm->red[1][c]) + (sm->red[2][c] + sm->red[3][c]);
                    sm->inv[c] = sum > 0.f ? 1.f / sum : (sum == sum ? 0.f : sum);
                    if (et < nc) {
                        if (whole)
                            p.lse[row0 + et] = sum > 0.f ? (sm->m_run[c] + log2f(sum)) * 0.69314718055994531f
                                                         : (sum == sum ? -INFINITY : sum);
                        else
                            p.part_ml[slot * p.slot_cols + c] = make_float2(sm->m_run[c], sum);
                    }
                }
                bar_sync(bar, 128);
                if (!mbar_wait(&sm->o_fin, seg & 1, kPtWait)) {
                    fail();
                    ok = false;
                }
                if (bar_red_or(bar, 128, !ok)) { ok = false; break; }
                tc_fence_after();
                uint64_t not_fin = 0;  // of rows that were made finite (rare)
                if (odd1 >= 0)
                    not_fin = hidden_values<ROWS == kBf16Rows ? NSA_DT_BF16 : NSA_DT_E4M3, kGrp>(
                        p.t.kv, p.t.num_pages, p.t.ps, pt, odd0, min(odd1, s.len - 1), sm->len + cb, key);
#pragma unroll 1
                for (int m = 0; m < 4; ++m) {
                    uint32_t v[kGrp];
                    tmem_ldg<kGrp>(lanes + m * NC + cb, v);
                    if (not_fin) {
#pragma unroll
                        for (int c = 0; c < kGrp; ++c)
                            if (not_fin >> (16 * m + c) & 1) v[c] = 0x7fffffffu;
                    }
                    __syncwarp();
                    if (whole) {
                        __nv_bfloat16 *o = p.out + row0 * kPtDl + m * 128 + key;
#pragma unroll
                        for (int c = 0; c < kGrp; ++c) {
                            const float r = __uint_as_float(v[c]) * sm->inv[cb + c];  // a column without a key: 0 times 0
                            if (c < nc) o[(int64_t)c * kPtDl] = __float2bfloat16_rn(r);
                        }
                    } else {
                        float *o = p.part + (slot * p.slot_cols + cb) * kPtDl + m * 128 + key;
#pragma unroll
                        for (int c = 0; c < kGrp; ++c)
                            if (c < nc) o[(int64_t)c * kPtDl] = __uint_as_float(v[c]);
                    }
                }
                tc_fence_before();
            }
        }
    } else if constexpr (RAW) {
        if (work) {
            // -------------------------------------------------------- raw rows expanded into the tile
            const int d = threadIdx.x - kRow0;
            uint32_t i = 0, rph = 0;
            int rs = 0;
            bool ok = true;
            for (bool more = true; more && ok; more = s.next(p, sm->share)) {
                for (int t = s.t0; t < s.t1 && ok; ++t, ++i) {
                    if (!mbar_wait(&sm->raw.tile_full[i & 1], (i >> 1) & 1, kPtWait)) ok = false;
                    const uint32_t live = live_rows(p.t, sm->raw.boxes[i & 1], d, t, s.len);
                    float *scales = reinterpret_cast<float *>(sc_s + (i & 1) * kScaleSlot);
#pragma unroll 1
                    for (int m = 0; m < 4; ++m) {
                        if (!mbar_wait(&sm->raw.full[rs], rph, kPtWait)) ok = false;
                        RawStep x;
                        x.read(raw_s + rs * kRawSlot, scales, m, d, live);
                        if constexpr (NC == 16) {  // expanded ahead of the wait (2 %); 32 columns leave no registers for it
                            uint4 e[kDqRows][2];
                            x.expand(e);
                            if (!mbar_wait(&sm->pair_free[m], (i & 1) ^ 1, kPtWait)) ok = false;
                            x.store(e, d, kv_s + 2 * m * kPtBlk, kv_s + (2 * m + 1) * kPtBlk);
                        } else {
                            if (!mbar_wait(&sm->pair_free[m], (i & 1) ^ 1, kPtWait)) ok = false;
                            x.store(d, kv_s + 2 * m * kPtBlk, kv_s + (2 * m + 1) * kPtBlk);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&sm->raw.empty[rs]);
                            mbar_arrive(&sm->pair_full[m]);
                        }
                        if (++rs == kRaw) {
                            rs = 0;
                            rph ^= 1;
                        }
                    }
                    ok = __all_sync(0xffffffffu, ok && !sm->abort) != 0;
                }
                ok = __all_sync(0xffffffffu, ok && !sm->abort) != 0;
            }
            if (!ok && lane == 0) fail();
        }
    } else if constexpr (SCR) {
        if (work) {
            // -------------------------------------------------------- rows expanded into the scratch
            const int d = threadIdx.x - kRow0;
            const int off = peer * kScrRows;     // this CTA's part of a tile
            constexpr int kSteps = kScrRows / kScrStep;  // steps a tile
            // The step whose page is asked for next: a step before its rows are loaded, which is two
            // steps before they are stored.  The page is looked at only then, so nothing waits for it
            // (a lookup in front of its loads took 2 - 3 thousand cycles a step).
            Seg f = s;
            int ft = f.t0, fu = 0, page = 0;
            int pos;  // of the row; -1: it holds no key, -2: there is no further step
            bool fetch = true;
            auto look = [&]() {
                pos = -2;
                if (!fetch) return;
                pos = ft * kPtTok + off + kScrStep * fu + (d >> 3);
                if (pos < f.len)
                    page = __ldg(p.t.page_table + (int64_t)f.b * p.t.pt_ld + pos / p.t.ps);
                else
                    pos = -1;
                if (++fu == kSteps) {
                    fu = 0;
                    if (++ft >= f.t1) {
                        fetch = f.next(p, sm->share);
                        ft = f.t0;
                    }
                }
            };
            int left = 0;  // steps loaded and not yet stored
            auto load = [&](ScrRows &x) {
                int slot = -1;
                if (pos != -2) ++left;
                if (pos >= 0) {
                    if (page >= 0 && page < p.t.num_pages)
                        slot = page * p.t.ps + pos % p.t.ps;
                    else
                        set_status(p.t.status, NSA_ERR_BOUNDS);
                }
                x.load(p.t, d, slot);
                look();
            };
            look();
            uint32_t n = 0;  // steps stored
            bool ok = true;
            auto step = [&](ScrRows &x) {
                const uint32_t tile = n / kSteps, u = n % kSteps, ss = tile % kScrSlots;
                if (u == 0 && tile >= kScrAhead) {
                    // This CTA has loaded tile - kScrAhead, and every CTA has written its part of it, which it does
                    // when it has loaded tile - 2 kScrAhead: nobody reads this slot any more.
                    const uint32_t s2 = (tile - kScrAhead) % kScrSlots, ph = (tile - kScrAhead) / kScrSlots & 1;
                    if (!mbar_wait(&sm->scr_loaded[s2], ph, kPtWait) || !mbar_wait_cluster(&sm->scr_full[s2], ph, kPtWait))
                        ok = false;
                }
                x.store(scr + ss * kScrTile, off + kScrStep * u + (d >> 3), d);
                --left;
                ++n;
                if (u == kSteps - 1) {
                    asm volatile("fence.proxy.async.global;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm->scr_part[ss]);
                    if (d == 0) sm->scr_tiles = tile + 1;
                }
                load(x);
                ok = __all_sync(0xffffffffu, ok && !sm->abort) != 0;
            };
            ScrRows x0, x1;
            load(x0);
            load(x1);
            while (left > 0 && ok) {
                step(x0);
                if (left > 0 && ok) step(x1);
            }
            if (!ok && lane == 0) fail();
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    if (CL > 1) cluster_sync_all();  // the peers' arrivals in this CTA are over
}

// Columns that several shares worked on: with M the largest maximum,
//   l = sum_q l_q 2^(m_q - M), out = sum_q O_q 2^(m_q - M) / l, lse = (M + log2 l) ln 2,
// in share order.  W warps a column (each a quarter, say, of the shares), 16 values of
// the latent a lane; one warp where requests are split in few shares, eight where one
// request is spread over the whole GPU.
constexpr int kJoinThreads = 256;

template <int W>
__global__ void __launch_bounds__(kJoinThreads) paged_mla_join_kernel(AParams p)
{
    __shared__ float4 acc_s[W > 1 ? W - 1 : 1][128];
    __shared__ float wl[W];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * (kJoinThreads / 32 / W) + warp / W;
    if (row >= (int64_t)p.t.B * p.cols) return;  // only with W == 1: whole warps leave, no barrier follows
    const int b = (int)(row / p.cols), c = (int)(row - (int64_t)b * p.cols);
    const int group = c / p.nc, set = group / p.team, rank = group - set * p.team, cc = c - group * p.nc;
    const int4 unit = p.unit[(int64_t)b * p.mult + set];  // its shares x .. y; z: share x started before it
    const int ns = unit.y - unit.x + 1;
    if (ns <= 1) return;  // one share had it whole, or there is no key (uniform over the block when W > 1)
    auto slot_of = [&](int q) -> int64_t {
        return (((int64_t)(unit.x + q) * p.team + rank) * 2 + (q == 0 ? unit.z : 0)) * p.slot_cols + cc;
    };
    float m = -INFINITY;
    for (int q = lane; q < ns; q += 32) m = fmaxf(m, p.part_ml[slot_of(q)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int part = W > 1 ? warp : 0, per = (ns + W - 1) / W, q0 = min(ns, part * per), q1 = min(ns, q0 + per);
    float4 acc[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 2
    for (int q = q0; q < q1; ++q) {
        const int64_t s = slot_of(q);
        const float2 ml = p.part_ml[s];
        const float4 *src = reinterpret_cast<const float4 *>(p.part + s * kPtDl) + lane;
        const float w = exp2f(ml.x - m);  // a share without a score: kNoMax, 0 and zeros (NaN for 0 x inf)
        l += w * ml.y;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float4 v = __ldcg(src + 32 * x);
            acc[x].x += w * v.x; acc[x].y += w * v.y; acc[x].z += w * v.z; acc[x].w += w * v.w;
        }
    }
    if constexpr (W > 1) {
        if (lane == 0) wl[part] = l;
        if (part > 0) {
#pragma unroll
            for (int x = 0; x < 4; ++x) acc_s[part - 1][lane + 32 * x] = acc[x];
        }
        __syncthreads();
        if (part > 0) return;
        l = 0.f;
        for (int w = 0; w < W; ++w) l += wl[w];
        for (int w = 0; w < W - 1; ++w) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float4 v = acc_s[w][lane + 32 * x];
                acc[x].x += v.x; acc[x].y += v.y; acc[x].z += v.z; acc[x].w += v.w;
            }
        }
    }
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    __nv_bfloat16 *o = p.out + row * kPtDl + 4 * lane;
    const bool wide = ((uintptr_t)p.out & 7) == 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const uint2 v = make_uint2(pack2(acc[x].x * inv, acc[x].y * inv), pack2(acc[x].z * inv, acc[x].w * inv));
        if (wide) {
            *reinterpret_cast<uint2 *>(o + 128 * x) = v;
        } else {
            const __nv_bfloat16 *e = reinterpret_cast<const __nv_bfloat16 *>(&v);
            for (int y = 0; y < 4; ++y) o[128 * x + y] = e[y];
        }
    }
    if (lane == 0) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : (l == l ? -INFINITY : l);
}

// Clusters of four scratch CTAs that the current device runs at once (asked once per device).
int clusters_of_four()
{
    constexpr int kMaxDev = 64;
    static std::atomic<int> cache[kMaxDev];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDev) {
        (void)cudaGetLastError();
        return 1;
    }
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
    constexpr auto kern = paged_mla_tc_kernel<kScratchRows, 4, kCols>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(4);
    cfg.blockDim = dim3(threads_of(kScratchRows, kCols));
    cfg.dynamicSmemBytes = smem_of(kScratchRows, kCols);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 4;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (max_dynamic_smem<kern>((int)cfg.dynamicSmemBytes) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();  // a failed query is not the caller's error
        return 1;
    }
    cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

// How the columns of a request are spread over CTAs: teams of the largest power of two
// up to kMaxTeam that divides the number of 64-column groups, as many as the SMs hold and
// the tiles fill.
struct Plan {
    Rows rows;
    int cluster;
    int cols, nc, groups, team, mult, teams, slot_cols;
    size_t head_bytes, ml_bytes, part_bytes, scratch_bytes;
};

Plan make_plan(bool fp8, int R, int n, int H, int max_row_len, int sms)
{
    Plan q;
    q.cols = n * H;
    q.nc = q.cols <= 16 ? 16 : q.cols <= 32 || (fp8 && q.cols <= kCols) ? 32 : kCols;
    q.groups = (int)ceil_div(q.cols, q.nc);
    q.rows = !fp8 ? kBf16Rows : q.cols <= 32 ? kRawRows : kScratchRows;
    if (q.rows == kScratchRows) q.groups = (q.groups + 1) / 2 * 2;  // pairs only: the last group may be padding
    q.team = 1;
    while (q.team < kMaxTeam && q.groups % (2 * q.team) == 0) q.team *= 2;
    q.mult = q.groups / q.team;
    // clusters of four halve what each CTA has to expand
    q.cluster = q.rows == kScratchRows ? (q.team >= 4 && q.nc == kCols ? 4 : 2) : 1;
    const int64_t most = (int64_t)(R / n) * q.mult * ceil_div(max_row_len, kPtTok);
    // the CTAs of a wave: clusters of four leave SMs of some GPCs idle
    const int ctas = q.cluster == 4 ? 4 * clusters_of_four() : sms;
    const int fit = ctas / q.team > 0 ? ctas / q.team : 1;
    q.teams = (int)(most < fit ? most : fit);
    q.slot_cols = q.cols < q.nc ? q.cols : q.nc;
    const size_t slots = (size_t)q.teams * q.team * 2 * q.slot_cols;
    q.head_bytes = (size_t)(R / n) * q.mult * sizeof(int4);
    q.ml_bytes = (slots * sizeof(float2) + 15) / 16 * 16;
    q.part_bytes = slots * kPtDl * sizeof(float);
    q.scratch_bytes = q.rows == kScratchRows ? (size_t)q.teams * q.team / q.cluster * scr_slots(q.cluster) * kScrTile : 0;
    return q;
}

struct Maps {
    CUtensorMap qn, qr, kv, sc, rope;
};

template <Rows ROWS, int CL, int NC>
nsa_status launch(const AParams &p, const Maps &m, cudaStream_t stream)
{
    constexpr auto kern = paged_mla_tc_kernel<ROWS, CL, NC>;
    constexpr int smem = (int)smem_of(ROWS, NC);
    NSA_CUDA_TRY(max_dynamic_smem<kern>(smem));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.teams * p.team));
    cfg.blockDim = dim3(threads_of(ROWS, NC));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    // bf16: pairs of a team side by side read a tile through the same part of L2 (169 -> 163 us, 32 x 128 heads)
    attr[0].val.clusterDim.x = ROWS == kBf16Rows && p.team % 2 == 0 ? 2 : CL;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    NSA_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, p, m.qn, m.qr, m.kv, m.sc, m.rope));
    // shares per request on average: below four, a warp joins a column faster than a block (both measured)
    if (p.teams == 1) return NSA_OK;  // every unit was one share's: nothing to join
    const int64_t rows = (int64_t)p.t.B * p.cols;
    const bool few = p.teams < 4 * (int64_t)p.t.B * p.mult;
    cudaLaunchConfig_t jc = {};
    jc.gridDim = dim3((unsigned)(few ? ceil_div(rows, kJoinThreads / 32) : rows));
    jc.blockDim = dim3(kJoinThreads);
    jc.stream = stream;
    attr[0] = pdl_attribute();
    jc.attrs = attr;
    jc.numAttrs = 1;
    NSA_CUDA_TRY(few ? cudaLaunchKernelEx(&jc, paged_mla_join_kernel<1>, p) : cudaLaunchKernelEx(&jc, paged_mla_join_kernel<8>, p));
    return NSA_OK;
}

}  // namespace

size_t paged_mla_tc_workspace_bytes(nsa_dtype q_dtype, nsa_dtype kv_dtype, int R, int rows_per_req, int H, int d_latent,
                                    int d_rope, int max_row_len)
{
    if (q_dtype != NSA_DT_BF16 || (kv_dtype != NSA_DT_BF16 && kv_dtype != NSA_DT_E4M3) || d_latent != kPtDl ||
        d_rope != kPtDr || R <= 0 || rows_per_req <= 0 || R % rows_per_req != 0 || H <= 0 || max_row_len <= 0 ||
        !paged_mla_sizes_ok(R, rows_per_req, H, max_row_len))
        return 0;
    // A bound on make_plan's sizes that grows with each argument, which they do not (fp8: clusters of four
    // need less scratch than pairs), so that a workspace for the largest shape of a loop serves all of it.
    const size_t units = (size_t)R * (size_t)ceil_div(H, 16);  // at least the group sets of all requests
    const size_t work = units * (size_t)ceil_div(max_row_len, kPtTok);
    const int sms = current_sm_count();
    const size_t most = (size_t)(sms > kMaxTeam ? sms : kMaxTeam), ctas = work < most ? work : most;
    const int64_t cols = (int64_t)rows_per_req * H;
    const size_t slots = ctas * 2 * (size_t)(cols < kCols ? cols : kCols);
    static_assert(scr_slots(2) >= scr_slots(4) / 2, "a CTA of a pair has the larger part of a scratch");
    return units * sizeof(int4) + (slots * sizeof(float2) + 15) / 16 * 16 + slots * kPtDl * sizeof(float) +
           (kv_dtype == NSA_DT_E4M3 && cols > 32 ? ctas * (scr_slots(2) / 2) * kScrTile : 0);
}

nsa_status paged_mla_tc_try_launch(const PagedMlaArgs &a, void *out, float *lse, void *workspace, size_t workspace_bytes,
                                   cudaStream_t stream)
{
    if (!paged_tc_applicable(a)) return NSA_ERR_UNSUPPORTED;
    const int sms = current_sm_count();
    if (sms <= 0) return NSA_ERR_CUDA;
    const bool fp8 = a.kv_dtype == NSA_DT_E4M3;
    const Plan q = make_plan(fp8, a.R, a.rows_per_req, a.H, a.max_row_len, sms);
    if (q.head_bytes + q.ml_bytes + q.part_bytes + q.scratch_bytes > workspace_bytes) return NSA_ERR_INVALID_ARG;
    if ((int64_t)(a.R / a.rows_per_req) * q.mult * (ceil_div(a.max_row_len, kPtTok) + piece_of(q.rows)) / q.teams >= kMaxShare)
        return NSA_ERR_UNSUPPORTED;
    AParams p;
    p.t = paged_tc_params(a);
    while (p.t.box_rows > kPtTok / q.cluster) p.t.box_rows /= 2;  // whole boxes for each CTA of a cluster
    p.cols = q.cols; p.nc = q.nc; p.groups = q.groups; p.team = q.team; p.mult = q.mult; p.teams = q.teams;
    p.slot_cols = q.slot_cols;
    p.out = (__nv_bfloat16 *)out;
    p.lse = lse;
    uint8_t *ws = (uint8_t *)workspace;
    p.unit = (int4 *)ws;
    p.part_ml = (float2 *)(ws += q.head_bytes);
    p.part = (float *)(ws += q.ml_bytes);
    p.scratch = ws += q.part_bytes;
    Maps m = {};
    if (!paged_tc_q_maps(a, (uint32_t)q.nc, &m.qn, &m.qr)) return NSA_ERR_CUDA;
    const bool mapped =
        q.rows == kBf16Rows ? bf16_rows_map(a.kv, (uint64_t)a.num_pages * a.page_size, (uint32_t)p.t.box_rows, &m.kv)
        : q.rows == kRawRows
            ? fp8_maps(a, (uint32_t)p.t.box_rows, 128, &m.kv, &m.sc, &m.rope)
            : true;
    if (!mapped) return NSA_ERR_CUDA;
    if (q.rows == kRawRows)
        return q.nc == 16 ? launch<kRawRows, 1, 16>(p, m, stream) : launch<kRawRows, 1, 32>(p, m, stream);
    if (q.rows == kScratchRows)
        return q.nc == 32          ? launch<kScratchRows, 2, 32>(p, m, stream)
               : q.cluster == 2 ? launch<kScratchRows, 2, 64>(p, m, stream)
                                : launch<kScratchRows, 4, 64>(p, m, stream);
    return q.nc == 16   ? launch<kBf16Rows, 1, 16>(p, m, stream)
           : q.nc == 32 ? launch<kBf16Rows, 1, 32>(p, m, stream)
                        : launch<kBf16Rows, 1, 64>(p, m, stream);
}

}  // namespace nsa
