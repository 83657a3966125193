// Pieces that the tensor-core kernels over a paged latent cache share
// (paged_mla_tc.cu, mla_key_weights_tc.cu): how the tiles of all requests are
// cut into equal shares, and how a tile of 128 cache rows reaches shared memory.
//
// A tile is 128 consecutive positions of one request as nine K-major blocks of
// 128 rows x 64 bf16 (16 KB, 128-byte swizzle): blocks 0..7 the latent, block 8
// the rope part.  bf16 rows come by TMA in boxes of box_rows rows x 64 columns
// that never cross a page; fp8 rows come raw and are expanded to bf16 by threads of the CTA.
#pragma once

#include "paged_mla.cuh"
#include "sm100_paged.cuh"
#include "tma_host.h"

namespace nsa {

constexpr int kPtTok = 128;                     // positions per tile
constexpr int kPtDl = 512, kPtDr = 64;
constexpr uint32_t kPtBlk = kPtTok * 128;       // bytes of a block
constexpr int kPtFp8Row = kPtDl + 16 + 2 * kPtDr;  // 656
constexpr long long kPtWait = 2000000000LL;     // ~1 s of SM clocks
constexpr int kDqThreads = 512;                 // fp8: threads that expand rows

struct PagedTc {
    const uint8_t *kv;
    int64_t num_pages;
    int ps, box_rows;
    const int32_t *page_table;
    int64_t pt_ld;
    const int32_t *row_len;
    int B, n, H, max_row_len;  // n rows per request
    float scale_log2;
    int32_t *status;
};

// The longest row of request b (0 for lengths out of range).
__device__ __forceinline__ int request_len(const PagedTc &p, int b)
{
    int len = 0;
    for (int i = 0; i < p.n; ++i) {
        const int L = p.row_len[(int64_t)b * p.n + i];
        if (L >= 0 && L <= p.max_row_len) len = max(len, L);
    }
    return len;
}

__device__ __forceinline__ int tiles_of(int len) { return (len + kPtTok - 1) / kPtTok; }

// Reports row lengths out of range (some threads of one CTA do it for the launch).
__device__ __forceinline__ void report_lengths(const PagedTc &p, int thread, int threads)
{
    for (int64_t r = thread; r < (int64_t)p.B * p.n; r += threads) {
        const int L = p.row_len[r];
        if (L < 0 || L > p.max_row_len) set_status(p.status, NSA_ERR_BOUNDS);
    }
}

// Where a share of the launch's work starts.  The tiles of all requests (each counted
// `mult` times, once for every unit of columns) lie in request order; in front of the tiles
// of a unit `piece` places are left for what starting and ending a unit costs a CTA.  These
// places are cut into up to `parts` equal shares; share `part` is [g0, g1) and begins at
// place `off` of request `b`.
struct TileShare {
    int64_t warp[32];
    int32_t units[32];
    unsigned long long later;    // of the requests that are not scanned at once
    int32_t later_units;
    int64_t total, g0, g1, off;  // total: places
    int b, len, piece, np;       // len: of request b; np: shares
};

__device__ __forceinline__ int64_t share_count(int64_t total, int parts)
{
    return total < 1 ? 1 : total < parts ? total : parts;
}

// total * k / np without a 64-bit division where the product fits 32 bits (shares of a decode
// step do; the long division costs a few hundred cycles of every CTA's start).
__device__ __forceinline__ int64_t share_start(int64_t total, int64_t k, int64_t np)
{
    const uint64_t x = (uint64_t)total * (uint64_t)k;
    return x < 0x100000000ULL ? (int64_t)((uint32_t)x / (uint32_t)np) : (int64_t)(x / (uint64_t)np);
}

__device__ __forceinline__ void find_share(const PagedTc &p, int mult, int max_piece, int part, int parts, TileShare *sh)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    const int n0 = blockDim.x;  // the first n0 requests are scanned, one a thread; more are rare
    auto len_of = [&](int b) { return b < p.B ? request_len(p, b) : 0; };
    const int len = len_of(tid);
    const int64_t v = (int64_t)tiles_of(len) * mult;
    const int c = v > 0 ? mult : 0;
    int64_t v_inc = v;
    int c_inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, v_inc, o);
        const int y = __shfl_up_sync(0xffffffffu, c_inc, o);
        if (lane >= o) {
            v_inc += x;
            c_inc += y;
        }
    }
    if (lane == 31) {
        sh->warp[warp] = v_inc;
        sh->units[warp] = c_inc;
    }
    if (p.B > n0) {
        if (tid == 0) {
            sh->later = 0;
            sh->later_units = 0;
        }
        __syncthreads();
        int64_t sum = 0;
        int units = 0;
        for (int b = n0 + tid; b < p.B; b += n0) {
            const int64_t x = (int64_t)tiles_of(len_of(b)) * mult;
            sum += x;
            units += x > 0 ? mult : 0;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            units += __shfl_xor_sync(0xffffffffu, units, o);
        }
        if (lane == 0) {
            atomicAdd(&sh->later, (unsigned long long)sum);
            atomicAdd(&sh->later_units, units);
        }
    }
    if (tid == 0) {
        sh->b = p.B;
        sh->off = 0;
    }
    __syncthreads();
    int64_t total = 0, units = 0, lo = 0, lo_units = 0;
    for (int w = 0; w < nw; ++w) {
        if (w == warp) {
            lo = total;
            lo_units = units;
        }
        total += sh->warp[w];
        units += sh->units[w];
    }
    const int64_t first = total, first_units = units;
    if (p.B > n0) {
        total += (int64_t)sh->later;
        units += sh->later_units;
    }
    // no more shares than tiles, and four times as many tiles as places of a piece in a share:
    // every share has a tile
    const int64_t np = share_count(total, parts);
    const int piece = (int)min((int64_t)max_piece, share_start(total, 1, 4 * np));
    total += piece * units;
    const int64_t g0 = part < np ? share_start(total, part, np) : total;
    const int64_t g1 = part < np ? share_start(total, part + 1, np) : total;
    if (tid == 0) {
        sh->total = total;
        sh->np = (int)np;
        sh->piece = piece;
        sh->g0 = g0;
        sh->g1 = g1;
    }
    lo += v_inc - v + piece * (lo_units + c_inc - c);
    const int64_t places = v + (int64_t)piece * c;
    if (g0 < g1 && places > 0 && g0 >= lo && g0 < lo + places) {
        sh->b = tid;
        sh->len = len;
        sh->off = g0 - lo;
    }
    int64_t before = first + piece * first_units;  // places of the requests below `base`
    for (int base = n0; base < p.B && g0 < g1 && before <= g0; base += n0) {
        __syncthreads();  // warp[] is free
        const int b = base + tid;
        const int l = len_of(b);
        const int64_t x = l > 0 ? (int64_t)(tiles_of(l) + piece) * mult : 0;
        int64_t inc = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) sh->warp[warp] = inc;
        __syncthreads();
        int64_t at = before, all = 0;
        for (int w = 0; w < nw; ++w) {
            if (w < warp) at += sh->warp[w];
            all += sh->warp[w];
        }
        at += inc - x;
        if (x > 0 && g0 >= at && g0 < at + x) {
            sh->b = b;
            sh->len = l;
            sh->off = g0 - at;
        }
        before += all;
    }
    __syncthreads();
}

// Page of position `pos` if the position is below `len` and its page exists, else -1.
__device__ __forceinline__ int checked_page(const PagedTc &p, const int32_t *pt, int pos, int len)
{
    if (pos >= len) return -1;
    const int page = __ldg(pt + pos / p.ps);
    if (page >= 0 && page < p.num_pages) return page;
    set_status(p.status, NSA_ERR_BOUNDS);
    return -1;
}

// ------------------------------------------------------------------ fp8 rows

// Four e4m3 codes (one word) times their block's scale as four bf16: code x scale rounded
// to fp32, then to bf16, the row's values by definition.
__device__ __forceinline__ uint2 expand4(uint32_t codes, float s)
{
    uint32_t h0, h1;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(h0), "=r"(h1)
        : "r"(codes));
    const float2 ss = make_float2(s, s);
    const float2 f0 = sm100::mul2(__half22float2(*reinterpret_cast<const __half2 *>(&h0)), ss);
    const float2 f1 = sm100::mul2(__half22float2(*reinterpret_cast<const __half2 *>(&h1)), ss);
    const __nv_bfloat162 b0 = __floats2bfloat162_rn(f0.x, f0.y), b1 = __floats2bfloat162_rn(f1.x, f1.y);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&b0), *reinterpret_cast<const uint32_t *>(&b1));
}

__device__ __forceinline__ uint4 expand8(uint32_t a, uint32_t b, float s)
{
    const uint2 x = expand4(a, s), y = expand4(b, s);
    return make_uint4(x.x, x.y, y.x, y.y);
}

// Raw fp8 rows in shared memory: the codes of one 128-value block of a tile's rows
// (128 x 128 bytes) a slot, loaded by TMA ahead of the threads that expand them, and
// the scales of a tile ([128][4] floats).  Plain 16-byte loads into registers reached
// 14 GB/s per SM from HBM; these boxes keep up with the SM's share of it.
constexpr uint32_t kRawSlot = kPtTok * 128;
constexpr uint32_t kScaleSlot = kPtTok * 16;
constexpr int kMaxRaw = 4;

struct RawShared {
    uint64_t full[kMaxRaw], empty[kMaxRaw];
    uint64_t tile_full[2];  // scales (and boxes) of the tile, by parity
    uint32_t boxes[2];      // boxes of the tile that were loaded
};

// Thread d of kDqThreads expands rows d / 8 and d / 8 + 64, chunk d % 8 (16 codes) of a
// step into blocks blk0 (chunks 0..3) and blk1; rows without a key become zeros.  Codes
// 16k .. 16k+15 become chunks 2k, 2k+1 of the step's 16.  Which of the two halves a lane
// takes first alternates with k / 4 and with the row, so that eight neighbouring lanes
// store to eight distinct bank groups and sixteen read distinct pairs of banks.  The
// arithmetic is what costs here (ncu: 61 % of issue slots, ALU 52 % busy, in an earlier
// form that chose the halves after loading them): two conversions, one paired multiply
// and two widenings for two codes.
// (Two groups of half the threads that take turns by steps were 7 - 9 % slower.)
constexpr int kDqRows = kPtTok * 8 / kDqThreads;
constexpr uint32_t kDqAll = (1u << kDqRows) - 1;

struct RawStep {
    uint2 w[kDqRows][2];
    float sc[kDqRows];

    static __device__ __forceinline__ bool swap(int d) { return ((d >> 2) ^ (d >> 3)) & 1; }

    __device__ __forceinline__ void read(uint8_t *raw, float *scales, int m, int d, uint32_t live)
    {
        uint8_t *at = raw + (d >> 3) * 128 + 16 * (d & 7);
        float *sp = scales + 4 * (d >> 3) + m;
        constexpr int kStep = kPtTok / kDqRows;  // rows between a thread's rows
        if (live != kDqAll) {
            // what an earlier tile left in the rows without a key may be NaN
#pragma unroll
            for (int u = 0; u < kDqRows; ++u)
                if (!(live >> u & 1)) {
                    *reinterpret_cast<uint4 *>(at + u * kStep * 128) = make_uint4(0u, 0u, 0u, 0u);
                    sp[u * kStep * 4] = 0.f;
                }
        }
        const int first = swap(d) ? 8 : 0;
#pragma unroll
        for (int u = 0; u < kDqRows; ++u) {
            w[u][0] = *reinterpret_cast<const uint2 *>(at + u * kStep * 128 + first);
            w[u][1] = *reinterpret_cast<const uint2 *>(at + u * kStep * 128 + (first ^ 8));
            sc[u] = sp[u * kStep * 4];
        }
    }
    // The same from rows of `pitch` bytes that hold more than the step's 128 codes (`raw` is the first
    // of them), with the rows' scales at hand.
    __device__ __forceinline__ void read_wide(uint8_t *raw, int pitch, const float (&scales)[kDqRows], int d, uint32_t live)
    {
        constexpr int kStep = kPtTok / kDqRows;
        uint8_t *at = raw + (d >> 3) * pitch + 16 * (d & 7);
        const int first = swap(d) ? 8 : 0;
#pragma unroll
        for (int u = 0; u < kDqRows; ++u) {
            if (!(live >> u & 1)) *reinterpret_cast<uint4 *>(at + u * kStep * pitch) = make_uint4(0u, 0u, 0u, 0u);
            w[u][0] = *reinterpret_cast<const uint2 *>(at + u * kStep * pitch + first);
            w[u][1] = *reinterpret_cast<const uint2 *>(at + u * kStep * pitch + (first ^ 8));
            sc[u] = scales[u];
        }
    }
    // The step's values, ahead of a wait for the blocks they go to.
    __device__ __forceinline__ void expand(uint4 (&e)[kDqRows][2]) const
    {
#pragma unroll
        for (int u = 0; u < kDqRows; ++u) {
            e[u][0] = expand8(w[u][0].x, w[u][0].y, sc[u]);
            e[u][1] = expand8(w[u][1].x, w[u][1].y, sc[u]);
        }
    }
    static __device__ __forceinline__ void store(const uint4 (&e)[kDqRows][2], int d, uint8_t *blk0, uint8_t *blk1)
    {
        const int k = d & 7, r = d >> 3, c0 = (2 * k) & 7, sw = swap(d) ? 1 : 0;
        uint8_t *blk = k < 4 ? blk0 : blk1;
        uint8_t *first = blk + sm100::sw128_offset(r, c0 + sw), *second = blk + sm100::sw128_offset(r, c0 + 1 - sw);
#pragma unroll
        for (int u = 0; u < kDqRows; ++u) {
            *reinterpret_cast<uint4 *>(first + u * (kPtTok / kDqRows) * 128) = e[u][0];
            *reinterpret_cast<uint4 *>(second + u * (kPtTok / kDqRows) * 128) = e[u][1];
        }
    }
    __device__ __forceinline__ void store(int d, uint8_t *blk0, uint8_t *blk1) const
    {
        const int k = d & 7, r = d >> 3, c0 = (2 * k) & 7, sw = swap(d) ? 1 : 0;
        uint8_t *blk = k < 4 ? blk0 : blk1;
        // rows 64 apart have the same swizzle
        uint8_t *first = blk + sm100::sw128_offset(r, c0 + sw), *second = blk + sm100::sw128_offset(r, c0 + 1 - sw);
#pragma unroll
        for (int u = 0; u < kDqRows; ++u) {
            *reinterpret_cast<uint4 *>(first + u * (kPtTok / kDqRows) * 128) = expand8(w[u][0].x, w[u][0].y, sc[u]);
            *reinterpret_cast<uint4 *>(second + u * (kPtTok / kDqRows) * 128) = expand8(w[u][1].x, w[u][1].y, sc[u]);
        }
    }
};
static_assert((kPtTok / kDqRows) % 8 == 0, "a thread's rows share their swizzle");

// The same for a step of 64 codes (slots of 128 x 64 bytes, one block a step), where shared
// memory is short: thread d expands chunk d % 4 of row d / 4.  Eight neighbouring lanes read
// 128 bytes in a row and store to eight distinct bank groups.
constexpr uint32_t kRawHalf = kPtTok * 64;

struct RawHalfStep {
    uint4 w;
    float sc;

    __device__ __forceinline__ void read(uint8_t *raw, float *scales, int m, int d, bool live)
    {
        uint4 *at = reinterpret_cast<uint4 *>(raw + 16 * d);
        float *sp = scales + 4 * (d >> 2) + (m >> 1);
        if (!live) {
            *at = make_uint4(0u, 0u, 0u, 0u);
            *sp = 0.f;
        }
        w = *at;
        sc = *sp;
    }
    __device__ __forceinline__ void store(int d, uint8_t *blk) const
    {
        const int r = d >> 2, c = 2 * (d & 3);
        *reinterpret_cast<uint4 *>(blk + sm100::sw128_offset(r, c)) = expand8(w.x, w.y, sc);
        *reinterpret_cast<uint4 *>(blk + sm100::sw128_offset(r, c + 1)) = expand8(w.z, w.w, sc);
    }
};
static_assert(kDqThreads == 4 * kPtTok, "a thread a chunk");

// Half rows: bytes 256 .. 527 (the codes from 256 on and the scales) and bytes 0 .. 255 of a tile's
// rows, a slot each.  TMA fetches a box row by row and a row line by line, and rows of 656 bytes lie
// across lines, so the fewer and longer the boxes' rows the better.
constexpr int kUpperRow = 256 + 16, kLowerRow = 256;
constexpr uint32_t kHalfRowSlot = kPtTok * kUpperRow;

// Which of thread d's rows of a tile hold a key (bit u: row d / 8 + 64 u).
__device__ __forceinline__ uint32_t live_rows(const PagedTc &p, uint32_t boxes, int d, int tile, int len)
{
    uint32_t live = 0;
#pragma unroll
    for (int u = 0; u < kDqRows; ++u) {
        const int r = (d >> 3) + kPtTok / kDqRows * u;
        if (tile * kPtTok + r < len && (boxes >> (r / p.box_rows) & 1)) live |= 1u << u;
    }
    return live;
}

// Rows expanded from registers into a scratch copy of the tile in global memory (which stays in
// L2), one copy a cluster: thread d of kScrThreads owns chunk d % 8 of each 128-value block of row
// d / 8 of a step's kScrStep.  The copy has the layout of the tile in shared memory (blocks of
// 128 x 128 bytes, swizzled), so that a pair of blocks comes from there as one run of bytes.  Two sets
// of registers take turns, so a row is loaded while the one before it is expanded.
constexpr int kScrThreads = 128;
constexpr int kScrStep = kScrThreads / 8;       // rows at a time
// Tiles that are expanded ahead of the loaded ones, by the cluster's size; a cluster's scratch holds
// twice as many.  Pairs expand four steps a tile and want to be told of a loaded tile at once, with a
// small scratch (32 x 128 heads: 256 us; three ahead 274).  Clusters of four expand two steps, which
// fit beside the next tile's first products: told only when the tile is done, three ahead, they
// stay out of the softmax's way (8 x 4 x 128 heads: 694 us; two ahead 772, told at once 777 - 793).
constexpr int scr_ahead(int cl) { return cl == 4 ? 3 : 2; }
constexpr int scr_slots(int cl) { return 2 * scr_ahead(cl); }
constexpr int kScrMaxSlots = scr_slots(4);
constexpr uint32_t kScrTile = 9 * kPtBlk;       // bytes of a tile's copy

struct ScrRows {
    uint4 w[5];
    float4 sc;

    // slot: the row's slot, or -1 for a row of zeros
    __device__ __forceinline__ void load(const PagedTc &p, int d, int slot)
    {
#pragma unroll
        for (int m = 0; m < 5; ++m) w[m] = make_uint4(0u, 0u, 0u, 0u);
        sc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (slot >= 0) {
            const uint8_t *row = p.kv + (int64_t)slot * kPtFp8Row;
#pragma unroll
            for (int m = 0; m < 5; ++m)
                w[m] = __ldg(reinterpret_cast<const uint4 *>(row + (m < 4 ? 128 * m : kPtDl + 16) + 16 * (d & 7)));
            sc = __ldg(reinterpret_cast<const float4 *>(row + kPtDl));
        }
    }
    // into row `row` of the tile's copy
    __device__ __forceinline__ void store(uint8_t *tile, int row, int d) const
    {
        const int k = d & 7;
        const float s[4] = {sc.x, sc.y, sc.z, sc.w};
        // codes 16k .. 16k+15 of a 128-value block become chunks 2k, 2k + 1 of its sixteen
        uint8_t *o0 = tile + (k >> 2) * kPtBlk + sm100::sw128_offset(row, (2 * k) & 7);
        uint8_t *o1 = tile + (k >> 2) * kPtBlk + sm100::sw128_offset(row, (2 * k + 1) & 7);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            *reinterpret_cast<uint4 *>(o0 + 2 * m * kPtBlk) = expand8(w[m].x, w[m].y, s[m]);
            *reinterpret_cast<uint4 *>(o1 + 2 * m * kPtBlk) = expand8(w[m].z, w[m].w, s[m]);
        }
        *reinterpret_cast<uint4 *>(tile + 8 * kPtBlk + sm100::sw128_offset(row, k)) = w[4];
    }
};

// ------------------------------------------------------------------ host

// One head per row: its rows follow one another at the row stride, whatever ld_h says.
inline PagedMlaArgs one_head_pitch(PagedMlaArgs a)
{
    if (a.H == 1 && a.R > 1) {
        a.nope_ld_h = a.nope_ld_r;
        a.rope_ld_h = a.rope_ld_r;
    }
    return a;
}

// Whether the tensor-core kernels take this problem: the 512 + 64 shape with bf16
// queries, whole boxes of 8 rows in a page, 16-byte aligned buffers and query rows
// that follow one another at one pitch (contiguous, or the two parts of a
// concatenated [R, H, 576] query).
inline bool paged_tc_applicable(const PagedMlaArgs &args)
{
    const PagedMlaArgs a = one_head_pitch(args);
    return a.q_dtype == NSA_DT_BF16 && (a.kv_dtype == NSA_DT_BF16 || a.kv_dtype == NSA_DT_E4M3) &&
           a.d_latent == kPtDl && a.d_rope == kPtDr && a.page_size % 8 == 0 && a.max_row_len > 0 &&
           (((uintptr_t)a.q_nope | (uintptr_t)a.q_rope | (uintptr_t)a.kv) & 15) == 0 && a.nope_ld_h % 8 == 0 &&
           a.rope_ld_h % 8 == 0 && a.nope_ld_h >= kPtDl && a.rope_ld_h >= kPtDr &&
           (a.R == 1 || (a.nope_ld_r == a.H * a.nope_ld_h && a.rope_ld_r == a.H * a.rope_ld_h));
}

inline PagedTc paged_tc_params(const PagedMlaArgs &a)
{
    PagedTc p;
    p.kv = (const uint8_t *)a.kv;
    p.num_pages = a.num_pages;
    p.ps = a.page_size;
    p.box_rows = kPtTok;
    while (a.page_size % p.box_rows != 0) p.box_rows /= 2;
    p.page_table = a.page_table;
    p.pt_ld = a.pt_ld;
    p.row_len = a.row_len;
    p.B = a.R / a.rows_per_req;
    p.n = a.rows_per_req;
    p.H = a.H;
    p.max_row_len = a.max_row_len;
    p.scale_log2 = a.sm_scale * 1.4426950408889634f;
    p.status = a.status;
    return p;
}

// Maps of the query parts: boxes of 64 columns x `rows` rows over the R * H query heads.
inline bool paged_tc_q_maps(const PagedMlaArgs &args, uint32_t rows, CUtensorMap *qn, CUtensorMap *qr)
{
    const PagedMlaArgs a = one_head_pitch(args);
    const uint64_t heads = (uint64_t)a.R * a.H;
    return make_tma_2d(qn, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q_nope, kPtDl, heads, (uint64_t)a.nope_ld_h * 2, 64, rows,
                       CU_TENSOR_MAP_SWIZZLE_128B) &&
           make_tma_2d(qr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q_rope, kPtDr, heads, (uint64_t)a.rope_ld_h * 2, 64, rows,
                       CU_TENSOR_MAP_SWIZZLE_128B);
}

// Map of the rows of a bf16 cache: boxes of 64 columns x box_rows rows.
inline bool bf16_rows_map(const void *base, uint64_t rows, uint32_t box_rows, CUtensorMap *kv)
{
    return make_tma_2d(kv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, kPtDl + kPtDr, rows, 2 * (kPtDl + kPtDr), 64, box_rows,
                       CU_TENSOR_MAP_SWIZZLE_128B);
}

// Maps of an fp8 cache: codes in boxes of box_codes bytes, scales in boxes of 16 bytes (the row
// seen as bytes) and the rope part in boxes of 64 bf16 (the row seen as 328 bf16; x = 264
// is byte 528, a multiple of 16).
inline bool fp8_maps(const PagedMlaArgs &a, uint32_t box_rows, uint32_t box_codes, CUtensorMap *codes, CUtensorMap *scales,
                     CUtensorMap *rope)
{
    const uint64_t rows = (uint64_t)a.num_pages * a.page_size;
    return make_tma_2d(codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.kv, kPtFp8Row, rows, kPtFp8Row, box_codes, box_rows,
                       CU_TENSOR_MAP_SWIZZLE_NONE) &&
           make_tma_2d(scales, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.kv, kPtFp8Row, rows, kPtFp8Row, 16, box_rows,
                       CU_TENSOR_MAP_SWIZZLE_NONE) &&
           make_tma_2d(rope, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.kv, kPtFp8Row / 2, rows, kPtFp8Row, 64, box_rows,
                       CU_TENSOR_MAP_SWIZZLE_128B);
}

// Maps of the half rows of an fp8 cache (the row seen as 164 words).
inline bool fp8_half_maps(const PagedMlaArgs &a, uint32_t box_rows, CUtensorMap *lower, CUtensorMap *upper, CUtensorMap *rope)
{
    const uint64_t rows = (uint64_t)a.num_pages * a.page_size;
    return make_tma_2d(lower, CU_TENSOR_MAP_DATA_TYPE_UINT32, a.kv, kPtFp8Row / 4, rows, kPtFp8Row, kLowerRow / 4, box_rows,
                       CU_TENSOR_MAP_SWIZZLE_NONE) &&
           make_tma_2d(upper, CU_TENSOR_MAP_DATA_TYPE_UINT32, a.kv, kPtFp8Row / 4, rows, kPtFp8Row, kUpperRow / 4, box_rows,
                       CU_TENSOR_MAP_SWIZZLE_NONE) &&
           make_tma_2d(rope, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.kv, kPtFp8Row / 2, rows, kPtFp8Row, 64, box_rows,
                       CU_TENSOR_MAP_SWIZZLE_128B);
}
constexpr int kUpperX = 256 / 4;  // word
constexpr int kFp8RopeX = (kPtDl + 16) / 2;
static_assert(kFp8RopeX * 2 % 16 == 0, "a TMA box starts on a 16-byte boundary");

}  // namespace nsa
