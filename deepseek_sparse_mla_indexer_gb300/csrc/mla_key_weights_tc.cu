// Tensor-core kernel of nsa_mla_key_weights for the 512 + 64 latent cache.
//
//   total[b, s] += sum_c 2^(x_{c,s} - lse2_c),   x = scale * log2(e) * (q_c . K_s)
//
// over the columns c = (row, head) of request b.  S[128 keys, N columns] =
// K_tile . Q^T accumulates in TMEM (tcgen05, bf16, fp32 accumulate), keys in the
// lanes: one epilogue thread owns one key and sums its columns in registers, so
// the sum over heads needs no exchange and runs in a fixed order.
//
// Each cache row is read once per pass over up to 128 columns, which is once for
// one row of 128 heads: 1152 (fp8: 656) bytes against 147 kflop a key, so the
// kernel is bound by HBM where one pass suffices.  More columns (verify) take several
// passes, made over four tiles at a time so that the tiles come from L2 after the
// first pass.
//
// One CTA per SM, persistent; the tiles of all requests are cut into equal shares.
// Roles: warp 0 issues TMA loads of Q and (bf16) of the tiles' blocks into a ring of
// 16 KB stages; warp 1 issues the MMAs into two TMEM buffers; warps 4..7 are the
// epilogue; fp8 rows come raw into slots of their own, from which warps 8..23 expand
// them into the ring (half rows up to 64 columns, blocks of 64 codes beyond, where Q
// leaves less room).
//
// Measured (GB300, a pass among others):
//   32 requests x 128 heads, bf16, 4096 .. 32768     97 us: 5.5 TB/s, 83 % of the copy rate
//   16 x 4 tokens x 16 heads, fp8, 16384 .. 65536   110 us: 3.5 TB/s
//   32 x 128 heads, fp8, 4096 .. 32768              127 us
//   2 x 16 heads, bf16, 700 and 2111                 13 us, the host's part of a call; 9 in a graph
// fp8 is bound by the chain of an expansion step (a wait, reads, conversions, stores, a proxy fence;
// issue slots 55 %): steps of 64 codes took 147 us where those of 128 take 110.
#include <cstddef>

#include "mla_key_weights_tc.cuh"
#include "paged_tc.cuh"

namespace nsa {
namespace {

using namespace sm100;

constexpr int kCols = 128;       // columns of one pass
constexpr int kMaxStages = 12;   // ring stages: as many as shared memory holds beside Q
constexpr int kPiece = 2;        // what a further request in a share costs, in tiles
constexpr int kPassTiles = 4;    // tiles per round of passes, when there are several
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kBufCols = 256;   // of one of the two score buffers
// A score is summed in four accumulators (two or three blocks of the row each) up to kSplitCols
// columns and in two beyond, which is what TMEM holds twice; the epilogue adds them.  The tensor
// core's accumulation truncates: a single chain of 36 products left scores 4.5e-7 of themselves
// too small, one-sided, and weights 1.6e-6 off (128 heads; two: 0.7e-6 at 1 % of the time).
constexpr int kSplitCols = 64;
constexpr float kLog2eLow = 1.92596299e-8f;  // log2(e) less its fp32 value

struct WShared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t q_full, q_empty, s_full[2], s_empty[2];
    RawShared raw;
    uint64_t rope_full, rope_empty;  // fp8: the rope parts have a stage of their own
    alignas(16) float nlse2[kCols];  // -lse in log2 units; -inf: no weight (padding, an empty row);
                                     // split scores: behind kSplitCols of them, the columns' factors
    int len[kCols];      // positions the column's row sees; 0: no weight
    int min_len[4];
    TileShare share;
    uint32_t tmem_base;
    volatile int abort;
};
constexpr size_t kAux = (sizeof(WShared) + 15) / 16 * 16;
static_assert(232448 - 1024 - 9 * kCols * 128 - kAux >= 5 * kPtBlk, "five stages beside 128 columns (four: 4 % slower)");

struct WParams {
    PagedTc t;
    const float *lse;
    float *total;
    int64_t total_ld;
    float scale_err;  // relative error of t.scale_log2
    int cols, passes, N, stages;  // columns per request, passes, MMA columns of a pass, ring stages
    int raw;                      // fp8: slots of raw codes
};

// The tiles of a share as (request, pass, tile range) pieces, the same for every role.
struct Walk {
    int b, t0, t1, c0, c1, pass, tiles, len, piece;
    int64_t left;  // places of the share behind tile t1

    __device__ __forceinline__ bool start(const WParams &p, const TileShare &s)
    {
        left = s.g1 - s.g0;
        if (left <= 0) return false;
        b = s.b;
        piece = s.piece;
        len = s.len;
        tiles = tiles_of(len);
        return enter(p, (int)s.off);
    }
    // the request from place `at` on; false if the share ends before its next tile
    __device__ __forceinline__ bool enter(const WParams &p, int at)
    {
        const int end = (int)min((int64_t)(tiles + piece), at + left);
        left -= end - at;
        t0 = max(0, at - piece);
        t1 = max(0, end - piece);
        c0 = t0;
        c1 = p.passes == 1 ? t1 : min(t1, c0 + kPassTiles);
        pass = 0;
        return t1 > t0;
    }
    __device__ __forceinline__ bool next(const WParams &p)
    {
        if (++pass < p.passes) return true;
        pass = 0;
        if (c1 < t1) {
            c0 = c1;
            c1 = min(t1, c0 + kPassTiles);
            return true;
        }
        if (left <= 0) return false;
        do {
            if (++b >= p.t.B) return false;
            len = request_len(p.t, b);
            tiles = tiles_of(len);
        } while (tiles == 0);
        return enter(p, 0);
    }
};

// SPLIT: scores in four accumulators (N <= kSplitCols).
template <bool FP8, bool SPLIT>
__global__ void __launch_bounds__(FP8 ? 256 + kDqThreads : 256, 1)
key_weights_tc_kernel(WParams p, const __grid_constant__ CUtensorMap qn_map, const __grid_constant__ CUtensorMap qr_map,
                      const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap sc_map,
                      const __grid_constant__ CUtensorMap rope_map)
{
    constexpr uint32_t kAccCols = SPLIT ? kSplitCols : kCols;
    constexpr bool HALF = FP8 && !SPLIT;  // Q leaves little shared memory: steps of 64 codes
    constexpr int kSteps = 8, kStepCodes = kPtDl / kSteps;  // of HALF
    constexpr bool WIDE = FP8 && SPLIT;   // else slots of half rows
    constexpr uint32_t kSlot = HALF ? kRawHalf : kHalfRowSlot;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *q_s = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t q_blk = (uint32_t)p.N * 128;
    uint8_t *ring = q_s + 9 * q_blk;
    uint8_t *rope_s = ring + (size_t)p.stages * kPtBlk;    // fp8: the rope part, raw codes, the scales of two tiles
    uint8_t *raw_s = rope_s + (FP8 ? kPtBlk : 0);
    uint8_t *sc_s = raw_s + (FP8 ? p.raw * kSlot : 0);
    WShared *sm = (WShared *)(sc_s + (HALF ? 2 * kScaleSlot : 0));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nst = p.stages;

    if (threadIdx.x == 0) {
        for (int i = 0; i < nst; ++i) {
            mbar_init(&sm->full[i], FP8 ? kDqThreads / 32 : 1);
            mbar_init(&sm->empty[i], 1);
        }
        for (int i = 0; i < kMaxRaw; ++i) {
            mbar_init(&sm->raw.full[i], 1);
            mbar_init(&sm->raw.empty[i], kDqThreads / 32);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&sm->raw.tile_full[i], 1);
        mbar_init(&sm->rope_full, 1);
        mbar_init(&sm->rope_empty, 1);
        mbar_init(&sm->q_full, 1);
        mbar_init(&sm->q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm->s_full[i], 1);
            mbar_init(&sm->s_empty[i], 128);
        }
        sm->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&sm->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    if (blockIdx.x == 0 && warp == 2) report_lengths(p.t, lane, 32);
    if (threadIdx.x == 96) {
        prefetch_tensormap(&qn_map);
        prefetch_tensormap(&qr_map);
        prefetch_tensormap(&kv_map);
    }
    tc_fence_before();
    find_share(p.t, 1, kPiece, blockIdx.x, gridDim.x, &sm->share);  // ends with a block barrier
    tc_fence_after();
    const uint32_t tmem = sm->tmem_base;
    auto fail = [&]() {
        sm->abort = 1;
        set_status(p.t.status, NSA_ERR_TIMEOUT);
    };
    Walk w;
    const bool work = w.start(p, sm->share);

    if (warp == 0) {
        // ------------------------------------------------------------ TMA
        if (work) {
            const int boxes = kPtTok / p.t.box_rows;  // at most 16, one a lane
            const uint32_t box_bytes = (uint32_t)p.t.box_rows * 128;
            int st = 0, rs = 0;
            uint32_t ph = 0, rph = 0, uses = 0, tile = 0;
            bool ok = true;
            for (bool more = true; more && ok; more = w.next(p)) {
                if (uses > 0 && !mbar_wait(&sm->q_empty, (uses - 1) & 1, kPtWait)) ok = false;
                const int row = w.b * p.cols + w.pass * kCols;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&sm->q_full, 9 * q_blk);
                    for (int c = 0; c < 8; ++c) tma_load_2d(q_s + c * q_blk, &qn_map, 64 * c, row, &sm->q_full);
                    tma_load_2d(q_s + 8 * q_blk, &qr_map, 0, row, &sm->q_full);
                }
                __syncwarp();
                ++uses;
                const int32_t *pt = p.t.page_table + (int64_t)w.b * p.t.pt_ld;
                auto box_row = [&](int t) -> int {  // row of this lane's box of tile t, or -1
                    const int pos = t * kPtTok + lane * p.t.box_rows;
                    const int page = lane < boxes && t < w.c1 ? checked_page(p.t, pt, pos, w.len) : -1;
                    return page < 0 ? -1 : page * p.t.ps + pos % p.t.ps;
                };
                int y = box_row(w.c0);
                for (int t = w.c0; t < w.c1 && ok; ++t, ++tile) {
                    const uint32_t live = __ballot_sync(0xffffffffu, y >= 0);
                    const uint32_t bytes = __popc(live) * box_bytes;
                    const int y_first = __shfl_sync(0xffffffffu, y, 0);
                    const int y_next = box_row(t + 1);  // its latency under this tile's waits
                    // the raw slots alone do not cover HBM's latency: a tile ahead into L2 (bf16 rows have
                    // the bytes in flight, and became a quarter slower from it)
                    if (FP8 && y_next >= 0)
                        prefetch_l2_bulk(p.t.kv + (int64_t)y_next * kPtFp8Row, (uint32_t)p.t.box_rows * kPtFp8Row);
                    // one lane issues a box at a time from uniform registers
                    auto boxes_of = [&](auto issue) {
                        int yb = y_first;
                        for (int x = 0; x < boxes; ++x) {
                            if (x > 0) yb = __shfl_sync(0xffffffffu, y, x);
                            if (yb >= 0 && elect_one()) issue(x, yb);
                            __syncwarp();
                        }
                    };
                    if constexpr (WIDE) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!mbar_wait(&sm->raw.empty[rs], rph ^ 1, kPtWait)) ok = false;
                            constexpr uint32_t kRow[2] = {kUpperRow, kLowerRow};
                            if (elect_one()) {
                                if (h == 0) sm->raw.boxes[tile & 1] = live;
                                mbar_arrive_expect_tx(&sm->raw.full[rs], bytes / 128 * kRow[h]);
                            }
                            __syncwarp();
                            boxes_of([&](int x, int yb) {
                                tma_load_2d(raw_s + rs * kSlot + x * p.t.box_rows * kRow[h], h == 0 ? &sc_map : &kv_map,
                                            h == 0 ? kUpperX : 0, yb, &sm->raw.full[rs]);
                            });
                            if (++rs == p.raw) {
                                rs = 0;
                                rph ^= 1;
                            }
                        }
                    } else if constexpr (HALF) {
                        for (int m = 0; m < kSteps; ++m) {
                            if (!mbar_wait(&sm->raw.empty[rs], rph ^ 1, kPtWait)) ok = false;
                            if (elect_one()) {
                                if (m == 0) {
                                    sm->raw.boxes[tile & 1] = live;
                                    mbar_arrive_expect_tx(&sm->raw.tile_full[tile & 1], bytes / 8);
                                }
                                mbar_arrive_expect_tx(&sm->raw.full[rs], bytes * kStepCodes / 128);
                            }
                            __syncwarp();
                            boxes_of([&](int x, int yb) {
                                tma_load_2d(raw_s + rs * kSlot + x * (box_bytes * kStepCodes / 128), &kv_map, kStepCodes * m, yb,
                                            &sm->raw.full[rs]);
                                if (m == 0)
                                    tma_load_2d(sc_s + (tile & 1) * kScaleSlot + x * (box_bytes / 8), &sc_map, kPtDl, yb,
                                                &sm->raw.tile_full[tile & 1]);
                            });
                            if (++rs == p.raw) {
                                rs = 0;
                                rph ^= 1;
                            }
                        }
                    } else {
                        for (int c = 0; c < 9; ++c) {
                            if (!mbar_wait(&sm->empty[st], ph ^ 1, kPtWait)) ok = false;
                            if (elect_one()) mbar_arrive_expect_tx(&sm->full[st], bytes);
                            __syncwarp();
                            boxes_of([&](int x, int yb) {
                                tma_load_2d(ring + st * kPtBlk + x * box_bytes, &kv_map, 64 * c, yb, &sm->full[st]);
                            });
                            if (++st == nst) {
                                st = 0;
                                ph ^= 1;
                            }
                        }
                    }
                    if constexpr (FP8) {
                        // the rope part straight into its stage
                        if (!mbar_wait(&sm->rope_empty, (tile & 1) ^ 1, kPtWait)) ok = false;
                        if (elect_one()) mbar_arrive_expect_tx(&sm->rope_full, bytes);
                        __syncwarp();
                        boxes_of([&](int x, int yb) {
                            tma_load_2d(rope_s + x * box_bytes, &rope_map, kFp8RopeX, yb, &sm->rope_full);
                        });
                    }
                    y = y_next;
                    ok = __all_sync(0xffffffffu, ok && !sm->abort) != 0;
                }
                ok = __all_sync(0xffffffffu, ok && !sm->abort) != 0;
            }
            if (!ok && lane == 0) fail();
            // nothing is in flight at the end: slots before st were filled last with phase ph, the others before
            if (lane == 0) {
                if (FP8) {
                    for (int i = 0; i < p.raw; ++i) mbar_wait(&sm->raw.full[i], i < rs ? rph : rph ^ 1, kPtWait);
                    if (tile > 0) mbar_wait(&sm->rope_full, (tile - 1) & 1, kPtWait);
                } else {
                    for (int i = 0; i < nst; ++i) mbar_wait(&sm->full[i], i < st ? ph : ph ^ 1, kPtWait);
                }
                if (HALF)
                    for (uint32_t x = tile > 2 ? tile - 2 : 0; x < tile; ++x)
                        mbar_wait(&sm->raw.tile_full[x & 1], (x >> 1) & 1, kPtWait);
                mbar_wait(&sm->q_full, (uses - 1) & 1, kPtWait);
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        // the whole warp walks and waits; one lane issues, with descriptors in uniform registers
        if (work) {
            const uint32_t idesc = instr_desc(1, 1, 0, 0, kPtTok, (uint32_t)p.N);
            const uint64_t q_desc = smem_desc(smem_u32(q_s), 16, 1024, kSwizzle128B);
            const uint64_t r_desc = smem_desc(smem_u32(ring), 16, 1024, kSwizzle128B);
            const uint64_t rope_desc = smem_desc(smem_u32(rope_s), 16, 1024, kSwizzle128B);
            int st = 0;
            uint32_t ph = 0, tile = 0, uses = 0;
            bool ok = true;
            for (bool more = true; more && ok; more = w.next(p)) {
                if (!mbar_wait(&sm->q_full, uses & 1, kPtWait)) ok = false;
                ++uses;
                for (int t = w.c0; t < w.c1 && ok; ++t, ++tile) {
                    const uint32_t buf = tile & 1, bph = (tile >> 1) & 1;
                    if (!mbar_wait(&sm->s_empty[buf], bph ^ 1, kPtWait)) ok = false;
                    for (int c = 0; c < 9; ++c) {
                        const bool rope = FP8 && c == 8;
                        const int qb = WIDE && !rope ? (c + 4) & 7 : c;  // the upper half of the row comes first
                        const int acc = SPLIT ? min(c >> 1, 3) : c >> 2 ? 1 : 0;
                        const bool first = SPLIT ? c < 8 && (c & 1) == 0 : c < 8 && (c & 3) == 0;
                        if (!mbar_wait(rope ? &sm->rope_full : &sm->full[st], rope ? tile & 1 : ph, kPtWait)) ok = false;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t a_desc = rope ? rope_desc : r_desc + st * (kPtBlk / 16);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_f16(tmem + buf * kBufCols + acc * kAccCols, a_desc + k * 2,
                                        q_desc + (qb * q_blk + k * 32) / 16, idesc, k > 0 || !first);
                            mma_commit(rope ? &sm->rope_empty : &sm->empty[st]);
                            if (c == 8) mma_commit(&sm->s_full[buf]);
                        }
                        __syncwarp();
                        if (!rope && ++st == nst) {
                            st = 0;
                            ph ^= 1;
                        }
                    }
                    ok = __all_sync(0xffffffffu, ok && !sm->abort) != 0;
                }
                if (elect_one()) mma_commit(&sm->q_empty);
                __syncwarp();
                ok = __all_sync(0xffffffffu, ok && !sm->abort) != 0;
            }
            if (!ok && lane == 0) fail();
            // the last commit tracks every MMA before it: nothing is in flight at the end
            mbar_wait(&sm->q_empty, (uses - 1) & 1, kPtWait);
            __syncwarp();
        }
    } else if (warp >= 4 && warp < 8) {
        // ------------------------------------------------------------ epilogue: one key a thread
        if (work) {
            const int key = threadIdx.x - 128;
            const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
            uint32_t tile = 0;
            bool more = true;
            while (more) {
                bar_sync(1, 128);  // the previous piece's columns are read out
                {
                    const int c = w.pass * kCols + key;
                    float nl = -INFINITY, fac = 1.f;
                    int len = 0;
                    if (c < p.cols) {
                        const int64_t r = (int64_t)w.b * p.t.n + c / p.t.H;
                        const float l = p.lse[r * p.t.H + c % p.t.H];
                        const int L = p.t.row_len[r];
                        if (l != -INFINITY && L > 0 && L <= p.t.max_row_len) {
                            // x - lse2 in log2 units with the rounded scale and lse2: what the scale's rounding
                            // takes from x (of about lse2 where the weight counts) goes into nl, and what nl then
                            // loses to its own rounding, up to 2^-20, into a factor near 1
                            const float nl0 = -l * 1.4426950408889634f;
                            const float lost = fmaf(l, 1.4426950408889634f, nl0) + l * kLog2eLow;
                            const float give = -fmaf(nl0, p.scale_err, lost);
                            nl = nl0 + give;
                            const float rest = give - (nl - nl0);
                            if (fabsf(rest) < 0.1f) fac = fmaf(rest, 0.69314718055994531f, 1.f);
                            len = L;
                        }
                    }
                    if (!SPLIT) {
                        sm->nlse2[key] = nl;
                    } else if (key < kSplitCols) {
                        sm->nlse2[key] = nl;
                        sm->nlse2[kSplitCols + key] = fac;
                    }
                    sm->len[key] = len;
                    // columns past the MMA's are never looked at
                    const int mn = __reduce_min_sync(0xffffffffu, key < p.N ? len : 0x7fffffff);
                    if (lane == 0) sm->min_len[warp & 3] = mn;
                }
                bar_sync(1, 128);
                const int min_len = min(min(sm->min_len[0], sm->min_len[1]), min(sm->min_len[2], sm->min_len[3]));
                const int32_t *pt = p.t.page_table + (int64_t)w.b * p.t.pt_ld;
                float *total = p.total + (int64_t)w.b * p.total_ld;
                for (int t = w.c0; t < w.c1; ++t, ++tile) {
                    const uint32_t buf = tile & 1, bph = (tile >> 1) & 1;
                    const int pos = t * kPtTok + key;
                    const bool valid = checked_page(p.t, pt, pos, w.len) >= 0;
                    const float old = valid ? total[pos] : 0.f;
                    const bool ok = mbar_wait(&sm->s_full[buf], bph, kPtWait);
                    if (!ok) fail();
                    if (bar_red_or(2, 128, !ok || sm->abort)) { more = false; break; }
                    tc_fence_after();
                    float sum = 0.f;
                    constexpr int kW = SPLIT ? 8 : 16;  // columns a step
                    auto scores = [&](int c0, uint32_t (&s)[kW]) {
                        const uint32_t at = lanes + buf * kBufCols + c0;
                        auto sum_of = [](uint32_t a, uint32_t b) {
                            return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
                        };
                        if constexpr (SPLIT) {
                            uint32_t u[3][kW];
                            tmem_ld8(at, s);
#pragma unroll
                            for (int a = 0; a < 3; ++a) tmem_ld8(at + (a + 1) * kAccCols, u[a]);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < kW; ++j) s[j] = sum_of(sum_of(s[j], u[0][j]), sum_of(u[1][j], u[2][j]));
                        } else {
                            uint32_t u[kW];
                            tmem_ld16(at, s);
                            tmem_ld16(at + kAccCols, u);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < kW; ++j) s[j] = sum_of(s[j], u[j]);
                        }
                    };
                    if ((t + 1) * kPtTok <= min_len) {
                        // every column is a real one and sees the whole tile: nothing to select
                        const float2 sc = make_float2(p.t.scale_log2, p.t.scale_log2);
                        const float4 *nl = reinterpret_cast<const float4 *>(sm->nlse2);
                        const float4 *fc = reinterpret_cast<const float4 *>(sm->nlse2 + kSplitCols);
                        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                        for (int c0 = 0; c0 < p.N; c0 += kW) {
                            uint32_t s[kW];
                            scores(c0, s);
#pragma unroll
                            for (int j = 0; j < kW / 4; ++j) {
                                const float4 n = nl[c0 / 4 + j];
                                float2 x = fma2(make_float2(__uint_as_float(s[4 * j]), __uint_as_float(s[4 * j + 1])), sc,
                                                make_float2(n.x, n.y));
                                float2 y = fma2(make_float2(__uint_as_float(s[4 * j + 2]), __uint_as_float(s[4 * j + 3])), sc,
                                                make_float2(n.z, n.w));
                                x = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                                y = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                                if constexpr (SPLIT) {
                                    const float4 f = fc[c0 / 4 + j];
                                    acc[0] = fma2(x, make_float2(f.x, f.y), acc[0]);
                                    acc[1] = fma2(y, make_float2(f.z, f.w), acc[1]);
                                } else {  // over more columns nl's roundings average out
                                    acc[0] = add2(acc[0], x);
                                    acc[1] = add2(acc[1], y);
                                }
                            }
                        }
                        sum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                    } else {
#pragma unroll 1
                        for (int c0 = 0; c0 < p.N; c0 += kW) {
                            uint32_t s[kW];
                            scores(c0, s);
#pragma unroll
                            for (int j = 0; j < kW; ++j) {
                                const float e = ex2_approx(fmaf(__uint_as_float(s[j]), p.t.scale_log2, sm->nlse2[c0 + j]));
                                // a column without weight may hold anything: selected away, not multiplied
                                const float v = pos < sm->len[c0 + j] ? e : 0.f;
                                sum = SPLIT ? fmaf(v, sm->nlse2[kSplitCols + c0 + j], sum) : sum + v;
                            }
                        }
                    }
                    tc_fence_before();
                    mbar_arrive(&sm->s_empty[buf]);
                    if (valid) total[pos] = old + sum;
                }
                if (more) more = w.next(p);
            }
        }
    } else if (FP8 && warp >= 8) {
        // ------------------------------------------------------------ raw rows expanded into the ring
        if (work) {
            const int d = threadIdx.x - 256;
            int st = 0, rs = 0;  // stage and raw slot of the step
            uint32_t ph = 0, rph = 0, tile = 0;
            bool ok = true;
            for (bool more = true; more && ok; more = w.next(p)) {
                for (int t = w.c0; t < w.c1 && ok; ++t, ++tile) {
                    if constexpr (HALF) {
                        if (!mbar_wait(&sm->raw.tile_full[tile & 1], (tile >> 1) & 1, kPtWait)) ok = false;
                        float *scales = reinterpret_cast<float *>(sc_s + (tile & 1) * kScaleSlot);
                        const uint32_t boxes = sm->raw.boxes[tile & 1];
                        const int r = d >> 2;
                        const bool live = t * kPtTok + r < w.len && (boxes >> (r / p.t.box_rows) & 1);
#pragma unroll 1
                        for (int m = 0; m < kSteps; ++m) {
                            if (!mbar_wait(&sm->raw.full[rs], rph, kPtWait)) ok = false;
                            RawHalfStep x;
                            x.read(raw_s + rs * kSlot, scales, m, d, live);
                            if (!mbar_wait(&sm->empty[st], ph ^ 1, kPtWait)) ok = false;
                            x.store(d, ring + st * kPtBlk);
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                mbar_arrive(&sm->raw.empty[rs]);
                                mbar_arrive(&sm->full[st]);
                            }
                            if (++st == nst) {
                                st = 0;
                                ph ^= 1;
                            }
                            if (++rs == p.raw) {
                                rs = 0;
                                rph ^= 1;
                            }
                        }
                    } else {
                        uint32_t live = 0;
                        float4 sc[kDqRows];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!mbar_wait(&sm->raw.full[rs], rph, kPtWait)) ok = false;
                            uint8_t *slot = raw_s + rs * kSlot;
                            if (h == 0) {
                                live = live_rows(p.t, sm->raw.boxes[tile & 1], d, t, w.len);
#pragma unroll
                                for (int u = 0; u < kDqRows; ++u) {
                                    const int r = (d >> 3) + u * (kPtTok / kDqRows);
                                    sc[u] = *reinterpret_cast<const float4 *>(slot + r * kUpperRow + 256);
                                    if (!(live >> u & 1)) sc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                                }
                            }
#pragma unroll
                            for (int m = 0; m < 2; ++m) {
                                const int s0 = st, s1 = st + 1 == nst ? 0 : st + 1;
                                const uint32_t ph0 = ph, ph1 = st + 1 == nst ? ph ^ 1 : ph;
                                st += 2;
                                if (st >= nst) {
                                    st -= nst;
                                    ph ^= 1;
                                }
                                float s[kDqRows];
#pragma unroll
                                for (int u = 0; u < kDqRows; ++u)
                                    s[u] = h == 0 ? (m == 0 ? sc[u].z : sc[u].w) : (m == 0 ? sc[u].x : sc[u].y);
                                RawStep x;
                                x.read_wide(slot + 128 * m, h == 0 ? kUpperRow : kLowerRow, s, d, live);
                                if (!mbar_wait(&sm->empty[s0], ph0 ^ 1, kPtWait)) ok = false;
                                if (!mbar_wait(&sm->empty[s1], ph1 ^ 1, kPtWait)) ok = false;
                                x.store(d, ring + s0 * kPtBlk, ring + s1 * kPtBlk);
                                fence_proxy_async_smem();
                                __syncwarp();
                                if (lane == 0) {
                                    if (m == 1) mbar_arrive(&sm->raw.empty[rs]);
                                    mbar_arrive(&sm->full[s0]);
                                    mbar_arrive(&sm->full[s1]);
                                }
                            }
                            if (++rs == p.raw) {
                                rs = 0;
                                rph ^= 1;
                            }
                        }
                    }
                    ok = __all_sync(0xffffffffu, ok && !sm->abort) != 0;
                }
                ok = __all_sync(0xffffffffu, ok && !sm->abort) != 0;
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
}

template <bool FP8, bool SPLIT>
nsa_status launch(const WParams &p, const CUtensorMap &qn, const CUtensorMap &qr, const CUtensorMap &kv,
                  const CUtensorMap &sc, const CUtensorMap &rope, unsigned grid, size_t smem, cudaStream_t stream)
{
    constexpr auto kern = key_weights_tc_kernel<FP8, SPLIT>;
    NSA_CUDA_TRY(max_dynamic_smem<kern>(232448));
    kern<<<grid, FP8 ? 256 + kDqThreads : 256, smem, stream>>>(p, qn, qr, kv, sc, rope);
    return launch_status();
}

}  // namespace

nsa_status key_weights_tc_try_launch(const PagedMlaArgs &a, const float *lse, float *total, int64_t total_ld,
                                     cudaStream_t stream)
{
    if (!paged_tc_applicable(a)) return NSA_ERR_UNSUPPORTED;
    const bool fp8 = a.kv_dtype == NSA_DT_E4M3;
    const int sms = current_sm_count();
    if (sms <= 0) return NSA_ERR_CUDA;
    WParams p;
    p.t = paged_tc_params(a);
    p.lse = lse;
    p.total = total;
    p.total_ld = total_ld;
    p.scale_err = (float)((double)a.sm_scale * 1.4426950408889634 / p.t.scale_log2 - 1.0);
    p.cols = a.rows_per_req * a.H;
    p.passes = (int)ceil_div(p.cols, kCols);
    p.N = p.passes > 1 ? kCols : (int)ceil_div(p.cols, 16) * 16;
    const size_t q_bytes = (size_t)9 * p.N * 128, left = 232448 - 1024 - kAux - q_bytes;
    // fp8: a stage for the rope part; of the rest two or three slots of half rows (a step fills two stages),
    // or with steps of 64 codes (one stage a step) three or four small ones
    const bool split = p.N <= kSplitCols, half = fp8 && !split;
    const size_t fixed = fp8 ? kPtBlk + (half ? 2 * kScaleSlot : 0) : 0, slot = half ? kRawHalf : kHalfRowSlot;
    const size_t rest = left - fixed;
    p.raw = !fp8 ? 0 : half ? (rest >= 8 * slot ? 4 : 3) : rest >= 3 * slot + 5 * kPtBlk ? 3 : 2;
    p.stages = (int)((rest - p.raw * slot) / kPtBlk);
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    const size_t smem = 1024 + q_bytes + fixed + p.raw * slot + (size_t)p.stages * kPtBlk + kAux;
    CUtensorMap qn, qr, kv, sc = {}, rope = {};
    if (!paged_tc_q_maps(a, (uint32_t)p.N, &qn, &qr)) return NSA_ERR_CUDA;
    if (half  ? !fp8_maps(a, (uint32_t)p.t.box_rows, 64, &kv, &sc, &rope)
        : fp8 ? !fp8_half_maps(a, (uint32_t)p.t.box_rows, &kv, &sc, &rope)
              : !bf16_rows_map(a.kv, (uint64_t)a.num_pages * a.page_size, (uint32_t)p.t.box_rows, &kv))
        return NSA_ERR_CUDA;
    const int64_t tiles = (int64_t)p.t.B * ceil_div(a.max_row_len, kPtTok);
    const unsigned grid = (unsigned)(tiles < sms ? tiles : sms);
    if (fp8) return split ? launch<true, true>(p, qn, qr, kv, sc, rope, grid, smem, stream)
                          : launch<true, false>(p, qn, qr, kv, sc, rope, grid, smem, stream);
    return split ? launch<false, true>(p, qn, qr, kv, sc, rope, grid, smem, stream)
                 : launch<false, false>(p, qn, qr, kv, sc, rope, grid, smem, stream);
}

}  // namespace nsa
