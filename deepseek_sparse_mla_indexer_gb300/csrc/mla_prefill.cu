// nsa_mla_prefill: attention of ragged prompts over expanded keys and values.  Per request, head h
// and query i, over the keys j that i sees (all n_k, or the first n_k - n_q + i + 1):
//   x_ij = sm_scale (q_nope[i,h] . k_nope[j,h] + q_rope[i,h] . k_rope[j])
//   lse  = ln sum_j exp(x_ij)        out = sum_j exp(x_ij - lse) v[j,h]
//
// A work item is 256 queries of one request and head, two tiles of 128, and a CTA (one an SM,
// persistent) takes one item after the other.  Per step of 128 keys and tile, on tcgen05:
//   S[128 q, 128 keys] = Q K^T        12 products, both operands in shared memory
//   P = 2^(c S - c m)                 256 threads, two a query; m a lazily refreshed maximum
//   O[128 q, 128]     += P V          8 products, P (bf16) in TMEM in the place of S
// S, P and O of both tiles fill TMEM (512 columns).  While 256 threads turn one tile's scores into
// P, the tensor core works on the other tile: PV of the step before, QK of the next.  A row's
// maximum is only refreshed, and O rescaled by the threads themselves, when a thread's 64 weights add up
// to more than 2^8: until then weights are up to 2^8 and nothing is lost, since sums are fp32.  So a
// step's weights are taken with the old maximum right away, and their sum, which is needed anyway, says
// afterwards whether that was right (one 8192-token prompt of 128 heads: 1598 us, and 1660 with every
// step's own maximum beside it).  Weights are rounded to bf16 (2^-8 of themselves at most) for the product
// with V, whose type the operands share; their sum, and so lse, is taken before that rounding.
//
// Keys and values come by TMA through a ring of eight 16 KB slots (a step takes five: two halves of
// the keys' nope part, the rope part that all heads share, and 64 keys' values each), Q has its own
// 96 KB.  One warp decodes the items from the sequences' starts, hands them out longest first per
// request, and issues the loads; one issues the products; two tell it what has landed.
//
// A value that is not finite, at a key that a query must not see, reaches that query as 0 x inf.  It
// shows in the result: an item whose last steps hide keys from some of its queries (causal diagonal,
// the end of a request inside a step) and whose result is not finite is done a second time, with
// care: such values are replaced by 0 in shared memory, and the queries that see them add them.  What
// they add needs no weights: with a positive one, whatever it is, a component becomes the value that is not
// finite (or NaN, from infinities of both signs), and a query sees a prefix of the keys.  So for a
// component the first key with each kind of such a value says all (every value NaN: 1238 us for 8192 tokens of 32 heads,
// 447 finite; one item of 256 tokens 110 us, 49 finite, and 15300 with weights taken again for each component).
//
// Few items (a short prompt over a long prefix, few heads) are cut along the keys; how often is
// chosen on the device, where the lengths are.  The parts' fp32 results go to the workspace, and
// merge_launch joins them.
//
// Measured (GB300, us in a graph on the same inputs / among passes whose inputs change; the latter of 1969 TFLOP/s):
//   one causal prompt of 8192, 128 heads       1556 - 1598 / 1725   1.59 PFLOP/s, 81 %
//   the same with 32 heads                      405 - 411 / -
//   eight prompts of 189 .. 2000, 128 heads     300 - 362 / 318     1.01, 51 % (1.20 with the hidden parts of the tiles)
//   1001 / 768 over 40000 / 26651, 16 heads     408 - 423 / 419     1.48, 75 %
//   37 after 600, 16 heads                      9.4 - 11.7 / 39: the host's part of the call
// (Ranges: between processes.)
// A step of both tiles takes 3170 cycles where its products alone take 2560: the tensor core reads
// shared memory at its full rate during QK (8 KB a product of 64 cycles), and the 80 KB that TMA writes a
// step come on top (640 cycles).  The long prompt runs at the power limit (1.9 GHz at 1375 W when
// repeated for seconds: 1.56 PFLOP/s).  Short prompts pay about 3.8 us an item beside its steps: the last
// step's softmax, which only one tile still has, the result's way out and the first step's softmax have no
// products beside them.
#include "mla_forms.cuh"

namespace nsa {
namespace {

using namespace sm100;

constexpr int kTile = 128;                 // queries of a tile, keys of a step
constexpr int kBlock = 2 * kTile;          // queries of an item
constexpr uint32_t kSlot = kTile * 128;    // 128 rows (K, Q) or 2 x 64 rows (V) of 128 bytes
constexpr int kSlots = 8;
constexpr int kKSlots = 3, kVSlots = 2, kStepSlots = kKSlots + kVSlots;
constexpr uint32_t kQTile = 3 * kSlot;

constexpr int kSoftmaxWarps = 16;          // per tile eight: two threads a query, 64 keys of a step each
constexpr int kHalf = kTile / 2;
constexpr int kLoadWarp = 16, kMmaWarp = 17, kScanWarp = 18, kScanWarps = 2;
constexpr int kThreads = 32 * (kScanWarp + kScanWarps);  // 20 warps: a 21st would leave each thread 80 registers instead of 96
constexpr uint32_t kTmemCols = 512;        // S of tile t at 128 t, each half's P in its first 32 columns; O at 256 + 128 t
constexpr long long kItemWait = 64 * kMlaWait;
constexpr float kJoinCost = 1.5f;           // steps
constexpr float kGrown = 256.0f;           // sum of a thread's weights that asks for a fresh maximum

// One work item, as the loading warp hands it to the others.
struct Item {
    int head;          // < 0: no more
    int rows;          // queries, 1 .. 256
    int64_t row0;      // of the first query
    int64_t key0;      // of the request's first key
    int keys;          // of the request
    int vis0;          // keys that the first query sees (causal: one more each further query); may be negative
    int j0, j1;        // steps of this share, none if j0 >= j1
    int n[2];          // steps that each tile needs at most
    int part, parts;   // of its request's keys
    int joined;        // parts that the join reads of each row; 0: the result is whole
    int careful;       // its masked steps' values are looked through (a second time for this item)
};

struct Shared {
    // of every other step: its keys / values have landed, and are no longer needed
    uint64_t k_full[2], v_full[2], k_free[2], v_free[2];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], go[2], o_full[2];  // go: P, and the values that it is multiplied with
    uint64_t item_full[2], item_empty[2];
    uint64_t drained;
    Item item[2];
    int again[2];                 // the item is to be done once more, with care
    int odd[2];                   // and then: some value of its masked steps is not finite
    uint32_t tmem;
    volatile int abort;
    // [tile][half]: a query's maximum over its half of the step, at the end its sum of weights, for the thread of
    // its other half
    float top[2][2][kTile];
};
constexpr uint32_t kSmem = 2 * kQTile + kSlots * kSlot + sizeof(Shared);
static_assert(kSmem <= 227 * 1024, "shared memory");

struct Params {
    const int32_t *cu_q, *cu_k;
    int B, total_q, total_k, H, causal;
    int heads_at_once;   // heads whose keys and values stay in L2 while all queries pass
    int most_blocks;     // of 256 queries, that requests in order have
    int most_parts;      // 1, or as many as the workspace holds
    int wide;            // the results' addresses are multiples of 32 bytes: out's (bit 0), the parts' (bit 1)
    float scale, scale_log2;
    // for the values that are not finite
    const __nv_bfloat16 *q_nope, *q_rope, *k_nope, *k_rope, *v;
    int64_t qn_r, qn_h, qr_r, qr_h, kn_r, kn_h, kr_r, v_r, v_h;
    __nv_bfloat16 *out;
    float *lse;
    float *part_out, *part_lse;  // [parts][total_q][H][128], [most_parts][total_q][H]
    int32_t *parts_used;         // for the join; NULL: most_parts is 1
    int *next;  // the items taken beyond each CTA's first; NULL: one each is all
    int32_t *status;
};

// Products whose operands' descriptors share the upper word: what issues them is on the tensor core's path, and
// adds one word instead of two.  A in shared memory; A in TMEM.
__device__ __forceinline__ void mma_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}"
        ::"r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_lo_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 bytes: one whole sector of L2 where the address allows it, since every thread of a warp writes a row of its own
// (past L1: one 8192-token prompt of 128 heads 1548 us, and 1555 through it).
__device__ __forceinline__ void store_sector(void *p, const uint32_t (&v)[8], bool wide)
{
    if (wide) {
        asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        *(uint4 *)p = make_uint4(v[0], v[1], v[2], v[3]);
        *((uint4 *)p + 1) = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// Queries and keys of request b; a request whose ranges are not in order is reported and has -1 queries (no block).
__device__ __forceinline__ int4 request(const Params &p, int b)
{
    const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
    if (q0 < 0 || q1 < q0 || q1 > p.total_q || k0 < 0 || k1 < k0 || k1 > p.total_k) {
        set_status(p.status, NSA_ERR_BOUNDS);
        return make_int4(0, -1, 0, 0);
    }
    return make_int4(q0, q1 - q0, k0, k1 - k0);
}

// The items a head that requests b0 .. b0 + 31 have up to and with this lane's.
__device__ __forceinline__ int scan_blocks(int blocks, int lane)
{
    for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, blocks, o);
        if (lane >= o) blocks += v;
    }
    return blocks;
}

// What a call has to do, from the sequences' starts.
struct Work {
    int units;       // items a head
    int parts;       // that the longest request's keys are cut into; 1: none are cut
    int share;       // steps of such a part; the other requests' are no longer (0: all requests have `parts`)
};

// Parts: where there are few items, or a few long ones, their keys are cut into shares.  What so many shares of a
// length cost, in units of a step (1.65 us): items of about one length go in rounds over the SMs; of different lengths,
// handed out longest first per request, they end within half a long one of each other where the long requests come
// first (requests go in the caller's order: a long last one ends up to a whole item behind the others).  An item takes two steps beside
// its own for its start and end; the join its launch and the fp32 results that it reads (`rows` of all parts; 0.12 us for
// 6 x 256 on 152 SMs; 0: there is no join).
__host__ __device__ inline float parts_cost(float items, int longest, float steps, float rows, float sms)
{
    const float share = longest + 2.f, even = (steps + 2.f * items) / sms;
    const float join = rows > 0.f ? kJoinCost + rows / (90.f * kBlock) : 0.f;
    if (items <= sms) return join + share;
    return join + (steps >= 0.8f * items * longest ? ceilf(items / sms) * share : fmaxf(share, even + 0.5f * share));
}

// Keys that block i of 256 queries of a request sees at most, in steps.
__host__ __device__ inline int block_steps(int nq, int nk, bool causal, int i)
{
    const int last = (i + 1) * kBlock < nq ? (i + 1) * kBlock : nq;
    const int vis = causal && nk - nq + last < nk ? nk - nq + last : nk;
    return vis > 0 ? (vis + kTile - 1) / kTile : 0;
}

__host__ __device__ inline int ceil_of(int a, int b) { return (a + b - 1) / b; }

// Parts of a request, from the steps of its longest block.
__device__ __forceinline__ int parts_of(const Work &todo, int longest)
{
    return todo.parts == 1 || todo.share == 0 ? todo.parts : max(1, ceil_of(longest, todo.share));
}

__device__ Work plan(const Params &p, int lane)
{
    int64_t n = 0, steps = 0, rows = 0;
    int longest = 0, first_blocks = 0, first_longest = 0;  // (of request `lane`)
    bool bad = false;
    for (int b = lane; b < p.B; b += 32) {
        const int4 r = request(p, b);
        const int blocks = ceil_of(r.y, kBlock);
        n += blocks;
        bad |= r.y < 0;
        if (p.most_parts == 1) continue;
        rows += r.y;
        for (int i = 0; i < blocks; ++i)  // few: the launch allows parts for few items alone
            steps += block_steps(r.y, r.w, p.causal, i);
        const int last = blocks > 0 ? block_steps(r.y, r.w, p.causal, blocks - 1) : 0;
        longest = max(longest, last);
        if (b == lane) {
            first_blocks = blocks;
            first_longest = last;
        }
    }
    for (int o = 16; o > 0; o /= 2) {
        n += __shfl_xor_sync(0xffffffffu, n, o);
        steps += __shfl_xor_sync(0xffffffffu, steps, o);
        rows += __shfl_xor_sync(0xffffffffu, rows, o);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (n > p.most_blocks) {  // requests that overlap: more items than the launch counted on
        if (lane == 0) set_status(p.status, NSA_ERR_BOUNDS);
        n = 0;
    }
    Work best = {(int)n, 1, 0};
    // (the join would write the rows of a request that is left out)
    if (n == 0 || __any_sync(0xffffffffu, bad)) return best;
    // All shares of about one length: a short request is cut into fewer than a long one (many requests, into as many)
    if (p.B == 1) {  // the launch knew the lengths
        best.parts = longest > 0 ? min(p.most_parts, longest) : 1;
        best.units = (int)n * best.parts;
        return best;
    }
    const float H = (float)p.H, sms = (float)gridDim.x;
    float cost = parts_cost((float)n * H, longest, (float)steps * H, 0.f, sms);
    for (int c = 2; c <= p.most_parts && c <= longest; ++c) {
        const int share = ceil_of(longest, c);
        const int units = p.B > 32 ? (int)n * c
                                   : __reduce_add_sync(0xffffffffu, first_blocks * max(1, ceil_of(first_longest, share)));
        const int parts = p.B > 32 ? c : ceil_of(longest, share);
        const float x = parts_cost((float)units * H, share, (float)steps * H, (float)rows * H * parts, sms);
        if (x < cost) {
            cost = x;
            best = {units, parts, p.B > 32 ? 0 : share};
        }
    }
    return best;
}

// Item w of units x H (below 2^31: the launch checks); first_requests: request `lane`, kept between
// calls.  Heads go in sections; in a section all heads of a block of queries follow one another, and a
// request's blocks go from its last, which sees most keys, to its first.
__device__ Item decode(const Params &p, int w, const Work &todo, int4 first_requests, int lane)
{
    Item it;
    const int per = todo.units * p.heads_at_once, section = w / per;
    w -= section * per;
    const int h0 = section * p.heads_at_once, hs = min(p.heads_at_once, p.H - h0);
    for (int b0 = 0;; b0 += 32) {
        const int b = b0 + lane;
        const int4 r = b0 == 0 ? first_requests : b < p.B ? request(p, b) : make_int4(0, 0, 0, 0);
        const int blocks = ceil_of(r.y, kBlock);
        const int parts = blocks > 0 && todo.parts > 1 ? parts_of(todo, block_steps(r.y, r.w, p.causal, blocks - 1)) : 1;
        const int upto = scan_blocks(blocks * parts, lane);
        const unsigned found = __ballot_sync(0xffffffffu, w / hs < upto);
        if (!found && b0 + 32 < p.B) {
            w -= __shfl_sync(0xffffffffu, upto, 31) * hs;
            continue;
        }
        const int src = found ? __ffs(found) - 1 : 0;  // found, unless the starts changed under the call
        const int q0 = __shfl_sync(0xffffffffu, r.x, src), nq = __shfl_sync(0xffffffffu, r.y, src);
        const int k0 = __shfl_sync(0xffffffffu, r.z, src), nk = __shfl_sync(0xffffffffu, r.w, src);
        const int nb = __shfl_sync(0xffffffffu, blocks, src);
        it.parts = __shfl_sync(0xffffffffu, parts, src);
        w -= (__shfl_sync(0xffffffffu, upto, src) - nb * it.parts) * hs;
        const int all = w / it.parts, block = all / hs;
        it.part = w - all * it.parts;
        it.head = h0 + (all - block * hs);
        const int first = max(0, nb - 1 - block) * kBlock;
        it.row0 = (int64_t)q0 + first;
        it.rows = found ? min(kBlock, nq - first) : 0;
        it.key0 = k0;
        it.keys = nk;
        it.vis0 = p.causal ? nk - nq + first + 1 : nk;
        break;
    }
    int all = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int rows = min(it.rows, kTile * (t + 1));  // the tile's last query sees most
        const int vis = p.causal ? min(it.keys, it.vis0 + rows - 1) : it.keys;
        it.n[t] = rows > kTile * t && vis > 0 ? (vis + kTile - 1) / kTile : 0;
        all = max(all, it.n[t]);
    }
    it.j0 = (int)((int64_t)all * it.part / it.parts);
    it.j1 = (int)((int64_t)all * (it.part + 1) / it.parts);
    it.joined = todo.parts > 1 ? todo.parts : 0;
    it.careful = 0;
    return it;
}

// The first step that some query of the item does not see wholly.
__device__ __forceinline__ int first_masked(const Item &it) { return max(it.vis0, 0) / kTile; }

// Where a query's result goes: 64 values from `col` on, times inv.
struct Place {
    void *dst;    // bf16 values of the result, or fp32 ones of a part
    float inv;
    bool whole, wide;
};

__device__ __forceinline__ Place place(const Params &p, const Item &it, int row, int col, float inv)
{
    const int64_t at = (it.row0 + row) * p.H + it.head;
    Place to;
    to.inv = inv;
    to.whole = it.joined == 0;
    to.wide = (p.wide & (to.whole ? 1 : 2)) != 0;
    to.dst = to.whole ? (void *)(p.out + at * kMlaV + col)
                      : (void *)(p.part_out + ((int64_t)it.part * p.total_q * p.H + at) * kMlaV + col);
    return to;
}

// Values 32 x .. of the 64.
__device__ __forceinline__ void store32(const Place &to, int x, const uint32_t (&o)[32])
{
    if (to.whole) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            uint32_t v[8];
#pragma unroll
            for (int z = 0; z < 8; ++z)
                v[z] = pack_bf16(__uint_as_float(o[16 * y + 2 * z]) * to.inv, __uint_as_float(o[16 * y + 2 * z + 1]) * to.inv);
            store_sector((__nv_bfloat16 *)to.dst + 32 * x + 16 * y, v, to.wide);
        }
    } else {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            uint32_t v[8];
#pragma unroll
            for (int z = 0; z < 8; ++z) v[z] = __float_as_uint(__uint_as_float(o[8 * y + z]) * to.inv);
            store_sector((float *)to.dst + 32 * x + 8 * y, v, to.wide);
        }
    }
}

// The result of a warp's queries (64 values from `col` on a thread, sums at o_at) where values at the keys from .. to - 1
// of the request, this share's masked steps, were taken out as not finite: the queries that see them (their first
// `vis` keys) add them here.
__device__ __noinline__ void rows_with_odd(const Params &p, const Item &it, int row, int vis, int from, int to, float l, int col,
                                           uint32_t o_at)
{
    // A lane looks through two components: the first key (counted from `from`) whose value is an infinity, with the sign
    // in the lowest bit, and the first one from which on the component is NaN
    const int lane = threadIdx.x % 32, none = 1 << 20;
    int pos[2] = {none, none}, neg[2] = {none, none}, nan[2] = {none, none}, inf[2];
    const __nv_bfloat16 *v = p.v + (it.key0 + from) * p.v_r + it.head * p.v_h + col + 2 * lane;
#pragma unroll 8
    for (int j = 0; j < to - from; ++j) {
        const uint32_t u = *(const uint32_t *)(v + j * p.v_r);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const uint32_t x = (y ? u : u << 16) & 0xFFFF0000u;
            if (x << 1 > 0xFF000000u) nan[y] = min(nan[y], j);
            if (x == 0x7F800000u) pos[y] = min(pos[y], j);
            if (x == 0xFF800000u) neg[y] = min(neg[y], j);
        }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        inf[y] = 2 * min(pos[y], neg[y]) + (neg[y] < pos[y] ? 1 : 0);
        nan[y] = min(nan[y], max(pos[y], neg[y]));
    }
    const Place to_row = place(p, it, row, col, l > 0.f ? 1.f / l : l == l ? 0.f : l);
    const int seen = vis - from;
#pragma unroll 1
    for (int x = 0; x < 2; ++x) {
        uint32_t o[32];
        tmem_ld32(o_at + 32 * x, o);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 32; ++c) {
            const int f = __shfl_sync(0xffffffffu, inf[c % 2], 16 * x + c / 2), n = __shfl_sync(0xffffffffu, nan[c % 2], 16 * x + c / 2);
            const uint32_t add = n < seen ? 0x7FC00000u : f & 1 ? 0xFF800000u : 0x7F800000u;
            // (added, since the steps that all queries see may have left an infinity too)
            if (n < seen || f / 2 < seen) o[c] = __float_as_uint(__uint_as_float(o[c]) + __uint_as_float(add));
            if (l == 0.f) o[c] = 0u;  // no weight at all: 0, and not 0 x NaN
        }
        if (row < it.rows) store32(to_row, x, o);
        __syncwarp();
    }
}

__global__ void __launch_bounds__(kThreads, 1)
mla_prefill_kernel(const __grid_constant__ CUtensorMap qn_map, const __grid_constant__ CUtensorMap qr_map,
                   const __grid_constant__ CUtensorMap kn_map, const __grid_constant__ CUtensorMap kr_map,
                   const __grid_constant__ CUtensorMap v_map, const __grid_constant__ Params p)
{
    extern __shared__ __align__(1024) uint8_t q_s[];
    uint8_t *ring = q_s + 2 * kQTile;
    Shared *sm = (Shared *)(ring + kSlots * kSlot);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        mbar_init(&sm->q_full, 1);
        mbar_init(&sm->q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm->k_full[i], 1);
            mbar_init(&sm->v_full[i], 1);
            mbar_init(&sm->k_free[i], 1);
            mbar_init(&sm->v_free[i], 1);
            mbar_init(&sm->s_full[i], 1);
            mbar_init(&sm->go[i], kSoftmaxWarps / 2 + kScanWarps);
            mbar_init(&sm->o_full[i], 1);
            mbar_init(&sm->item_full[i], 1);
            mbar_init(&sm->item_empty[i], kSoftmaxWarps + 1 + kScanWarps);
        }
        mbar_init(&sm->drained, 1);
        sm->abort = 0;
        sm->again[0] = sm->again[1] = 0;
        fence_mbar_init();
        prefetch_tensormap(&qn_map);
        prefetch_tensormap(&qr_map);
        prefetch_tensormap(&kn_map);
        prefetch_tensormap(&kr_map);
        prefetch_tensormap(&v_map);
    }
    if (warp == kMmaWarp) tmem_alloc(&sm->tmem, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm->tmem;
    volatile int *abort = &sm->abort;
    bool ok = true;
    pdl_wait();  // every warp, so that no bounded wait counts the time of the launch before this one

    // Item i as the loading warp published it; its place is given back with item_done.
    // (Warps without work in an item wait for the next one as long as it takes.)
    const auto item_wait = [&](int i) { return mla_wait(&sm->item_full[i & 1], (i >> 1) & 1, abort, kItemWait); };
    const auto item_done = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->item_empty[i & 1]);
    };

    if (warp == kLoadWarp) {
        // ------------------------------------------------------------ items and loads
        const Work todo = plan(p, lane);
        const int total = todo.units * p.H;
        const int4 first_requests = lane < p.B ? request(p, lane) : make_int4(0, 0, 0, 0);
        if (p.parts_used && blockIdx.x == 0 && lane == 0) *p.parts_used = todo.parts;
        uint32_t g = 0, q_uses = 0;  // steps and Q buffers filled so far
        int w = blockIdx.x;
        Item next;
        next.head = -1;
        if (w < total) next = decode(p, w, todo, first_requests, lane);
        // K of step g takes the slots of K (its last) and V of step g - 2, V those of K of step g - 1
        uint32_t k_sent = 0, v_sent = 0;
        const auto load_k = [&](const Item &it, int j) {
            if (!ok) return;
            const int r = (int)it.key0 + j * kTile;
            uint64_t *bar = &sm->k_full[g & 1];
            const auto slot = [&](int x) { return ring + (kStepSlots * g + x) % kSlots * kSlot; };
            mbar_arrive_expect_tx(bar, kKSlots * kSlot);
            ++k_sent;
            tma_load_3d(slot(0), &kn_map, 0, it.head, r, bar);
            if (g >= 2) ok = mla_wait(&sm->v_free[g & 1], ((g - 2) >> 1) & 1, abort);
            // (given up or not: what the barrier expects is sent)
            tma_load_3d(slot(1), &kn_map, 64, it.head, r, bar);
            tma_load_2d(slot(2), &kr_map, 0, r, bar);
        };
        const auto load_v = [&](const Item &it, int j) {
            const int r = (int)it.key0 + j * kTile;
            uint64_t *bar = &sm->v_full[g & 1];
            if (g >= 1) ok = ok && mla_wait(&sm->k_free[(g - 1) & 1], ((g - 1) >> 1) & 1, abort);
            if (!ok) return;
            mbar_arrive_expect_tx(bar, kVSlots * kSlot);
            ++v_sent;
            for (int x = 0; x < kVSlots; ++x) {
                uint8_t *dst = ring + (kStepSlots * g + kKSlots + x) % kSlots * kSlot;
                tma_load_3d(dst, &v_map, 0, it.head, r + 64 * x, bar);
                tma_load_3d(dst + kSlot / 2, &v_map, 64, it.head, r + 64 * x, bar);
            }
        };
        for (int i = 0; ok; ++i) {
            ok = __all_sync(0xffffffffu, mla_wait(&sm->item_empty[i & 1], ((i >> 1) & 1) ^ 1, abort, kItemWait));
            // (behind the last item, the one in the other place may still ask to be done again)
            if (ok && next.head < 0 && !sm->again[i & 1] && i > 0) {
                ok = __all_sync(0xffffffffu, mla_wait(&sm->item_empty[(i - 1) & 1], ((i - 1) >> 1) & 1, abort, kItemWait));
            }
            if (!ok) break;
            const bool mine = sm->again[i & 1], other = next.head < 0 && sm->again[(i & 1) ^ 1], again = mine || other;
            Item it = again ? sm->item[mine ? i & 1 : (i & 1) ^ 1] : next;
            __syncwarp();
            if (again) it.careful = 1;
            if (lane == 0) {
                sm->odd[i & 1] = 0;
                sm->again[mine ? i & 1 : other ? (i & 1) ^ 1 : i & 1] = 0;
            }
            __syncwarp();
            if (lane == 0) {
                sm->item[i & 1] = it;
                mbar_arrive(&sm->item_full[i & 1]);
            }
            if (it.head < 0) break;
            const bool some = it.j0 < it.j1;
            if (some && lane == 0) {
                load_k(it, it.j0);
                ok = ok && mla_wait(&sm->q_empty, (q_uses & 1) ^ 1, abort);
                if (ok) {
                    const int tiles = it.rows > kTile ? 2 : 1;
                    mbar_arrive_expect_tx(&sm->q_full, tiles * kQTile);
                    for (int t = 0; t < tiles; ++t) {
                        uint8_t *q = q_s + t * kQTile;
                        const int r = (int)it.row0 + t * kTile;
                        tma_load_3d(q, &qn_map, 0, it.head, r, &sm->q_full);
                        tma_load_3d(q + kSlot, &qn_map, 64, it.head, r, &sm->q_full);
                        tma_load_3d(q + 2 * kSlot, &qr_map, 0, it.head, r, &sm->q_full);
                    }
                    ++q_uses;
                }
                load_v(it, it.j0);
                ++g;
            }
            // the item after this one is looked up while this one's steps run
            if (again) {
                // (the next one waits)
            } else if (p.next) {
                int n = 0;
                if (lane == 0) n = atomicAdd(p.next, 1);
                w = gridDim.x + __shfl_sync(0xffffffffu, n, 0);
            } else {
                w += gridDim.x;
            }
            if (!again) {
                next.head = -1;
                if (w < total) next = decode(p, w, todo, first_requests, lane);
            }
            if (some && lane == 0) {
                for (int j = it.j0 + 1; j < it.j1 && ok; ++j, ++g) {
                    load_k(it, j);
                    load_v(it, j);
                }
            }
            ok = __all_sync(0xffffffffu, ok);
        }
        if (!ok && lane == 0) {
            set_status(p.status, NSA_ERR_TIMEOUT);
            // copies in flight end before the block does
            for (uint32_t x = k_sent > 2 ? k_sent - 2 : 0; x < k_sent; ++x) mbar_wait(&sm->k_full[x & 1], (x >> 1) & 1, kMlaWait);
            for (uint32_t x = v_sent > 2 ? v_sent - 2 : 0; x < v_sent; ++x) mbar_wait(&sm->v_full[x & 1], (x >> 1) & 1, kMlaWait);
            if (q_uses > 0) mbar_wait(&sm->q_full, (q_uses - 1) & 1, kMlaWait);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ products
        const uint32_t idesc_s = instr_desc(1, 1, 0, 0, kTile, kTile);   // K-major both
        const uint32_t idesc_o = instr_desc(1, 1, 0, 1, kTile, kMlaV);   // P in TMEM, V MN-major
        const uint64_t q_desc = smem_desc(smem_u32(q_s), 16, 1024, kSwizzle128B);
        const uint64_t k_desc = smem_desc(smem_u32(ring), 16, 1024, kSwizzle128B);
        const uint64_t v_desc = smem_desc(smem_u32(ring), kSlot / 2, 1024, kSwizzle128B);
        const uint32_t k_hi = (uint32_t)(k_desc >> 32), v_hi = (uint32_t)(v_desc >> 32);  // (q_desc's is k_desc's)
        // What this warp does between products leaves the tensor core without work, so one barrier a tile and
        // step tells it that P and V are there
        uint32_t g = 0, q_uses = 0, go_uses[2] = {0, 0};
        // a wait that gave up lets the warp go on to the step's end, where the lanes agree to stop
        const auto wait = [&](uint64_t *bar, uint32_t parity) { ok = mla_wait(bar, parity, abort) && ok; };
        // (one elected lane) S_t = Q_t K^T, O_t += P_t V, K and V of this CTA's step `at`
        const auto qk = [&](int t, uint32_t at) {
#pragma unroll
            for (int x = 0; x < kKSlots; ++x) {
                const uint32_t a = (uint32_t)q_desc + (t * kQTile + x * kSlot) / 16;
                const uint32_t b = (uint32_t)k_desc + (kStepSlots * at + x) % kSlots * (kSlot / 16);
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_lo(tmem + t * kTile, a + 2 * k, b + 2 * k, k_hi, idesc_s, x > 0 || k > 0);
            }
            mma_commit(&sm->s_full[t]);
        };
        const auto pv = [&](int t, uint32_t at, bool first, bool last) {
#pragma unroll
            for (int x = 0; x < kVSlots; ++x) {
                const uint32_t b = (uint32_t)v_desc + (kStepSlots * at + kKSlots + x) % kSlots * (kSlot / 16);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_lo_ts(tmem + 2 * kTile + t * kMlaV, tmem + t * kTile + x * kHalf + k * 8, b + k * (2048 / 16), v_hi, idesc_o,
                              !first || x > 0 || k > 0);
            }
            if (last) mma_commit(&sm->o_full[t]);
        };
        for (int i = 0; ok; ++i) {
            ok = __all_sync(0xffffffffu, item_wait(i));
            if (!ok) break;
            const int head = sm->item[i & 1].head, j0 = sm->item[i & 1].j0, j1 = sm->item[i & 1].j1;
            const int n[2] = {sm->item[i & 1].n[0], sm->item[i & 1].n[1]};
            item_done(i);
            if (head < 0) break;
            if (j0 >= j1) continue;
            wait(&sm->k_full[g & 1], (g >> 1) & 1);
            wait(&sm->q_full, q_uses++ & 1);
            __syncwarp();
            if (elect_one()) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (j0 < n[t]) qk(t, g);
                mma_commit(&sm->k_free[g & 1]);
                if (j1 - j0 == 1) mma_commit(&sm->q_empty);  // behind the item's last product with Q
            }
            for (int j = j0; j < j1; ++j) {
                const bool more = j + 1 < j1;
                bool have_k = more && mbar_test(&sm->k_full[(g + 1) & 1], ((g + 1) >> 1) & 1);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (j < n[t]) {
                        wait(&sm->go[t], go_uses[t]++ & 1);
                        __syncwarp();
                        tc_fence_after();
                    }
                    if (elect_one()) {
                        if (j < n[t]) pv(t, g, j == j0, !(more && j + 1 < n[t]));
                        if (t == 1) mma_commit(&sm->v_free[g & 1]);
                    }
                    if (t == 0 && more && !have_k) wait(&sm->k_full[(g + 1) & 1], ((g + 1) >> 1) & 1);
                    __syncwarp();
                    if (elect_one()) {
                        if (more && j + 1 < n[t]) qk(t, g + 1);
                        if (t == 1 && more) mma_commit(&sm->k_free[(g + 1) & 1]);
                        if (t == 1 && j + 2 == j1) mma_commit(&sm->q_empty);
                    }
                    __syncwarp();
                }
                ++g;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
            }
        }
        if (!ok && lane == 0) {
            set_status(p.status, NSA_ERR_TIMEOUT);
            mma_commit(&sm->drained);  // products in flight end before the block does
            mbar_wait(&sm->drained, 0, kMlaWait);
        }
        __syncwarp();
    } else if (warp >= kScanWarp) {
        // ------------------------------------------------------------ what has landed, for the products
        // A step's values; those that some queries must not see are looked through
        uint32_t g = 0;
        for (int i = 0; ok; ++i) {
            ok = __all_sync(0xffffffffu, item_wait(i));
            if (!ok) break;
            const Item it = sm->item[i & 1];
            if (it.head < 0) break;
            const int masked = first_masked(it);
            for (int j = it.j0; j < it.j1 && ok; ++j, ++g) {
                ok = __all_sync(0xffffffffu, mla_wait(&sm->v_full[g & 1], (g >> 1) & 1, abort));
                const auto go = [&] {
                    // behind the products of the step before, so that its `go` is over
                    if (g > 0) ok = ok && mla_wait(&sm->v_free[(g - 1) & 1], ((g - 1) >> 1) & 1, abort);
                    __syncwarp();
                    if (lane < 2 && j < it.n[lane]) mbar_arrive(&sm->go[lane]);
                };
                if (j < masked || !it.careful) {
                    go();
                    continue;
                }
                // a slot has 64 keys' rows of 128 bytes, one half of the value behind the other; eight lanes a row
                for (int x = warp - kScanWarp; x < kVSlots && ok; x += kScanWarps) {
                    uint8_t *slot = ring + (kStepSlots * g + kKSlots + x) % kSlots * kSlot;
                    const uint32_t at0 = smem_u32(slot) + lane * 16;
                    uint32_t seen = 0;
                    // an exponent of ones carries into the sign's place
#pragma unroll 8
                    for (int r = 0; r < 2 * 64; r += 4) {
                        uint32_t u[4];
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(at0 + r * 128));
#pragma unroll
                        for (int y = 0; y < 4; ++y) seen |= (u[y] & 0x7FFF7FFFu) + 0x00800080u;
                    }
                    if (!__any_sync(0xffffffffu, seen & 0x80008000u)) continue;
                    for (int r = 0; r < 2 * 64; r += 4) {
                        uint4 *at = (uint4 *)(slot + (r + lane / 8) * 128 + (lane % 8) * 16);
                        uint4 v = *at;
                        uint32_t *u = &v.x;
                        bool any = false;
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const bool lo = (u[y] & 0x7F80u) == 0x7F80u, hi = (u[y] & 0x7F800000u) == 0x7F800000u;
                            if (lo) u[y] &= 0xFFFF0000u;
                            if (hi) u[y] &= 0x0000FFFFu;
                            any |= lo || hi;
                        }
                        if (any) *at = v;
                    }
                    if (lane == 0) sm->odd[i & 1] = 1;
                    fence_proxy_async_smem();
                }
                go();
            }
            item_done(i);
        }
        if (!ok && lane == 0) set_status(p.status, NSA_ERR_TIMEOUT);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax: two threads a query, 64 keys each
        const int t = (warp / 4) & 1, half = warp / 8, row = (warp & 3) * 32 + lane;  // of tile t
        const int two = 1 + t * 4 + (warp & 3);  // the barrier of the two warps that share their queries
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_at = lanes + t * kTile + half * kHalf;
        const uint32_t o_at = lanes + 2 * kTile + t * kMlaV + half * kHalf;
        uint32_t s_uses = 0, o_uses = 0;
        const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
        for (int i = 0;; ++i) {
            // The two warps of a row meet at barriers, so they give up together: where a wait ran out they go on to
            // here (the waits that follow return at once)
            ok = item_wait(i) && ok;
            __syncwarp();
            if (bar_red_or(two, 64, !ok)) {
                ok = false;
                break;
            }
            const Item &it = sm->item[i & 1];
            if (it.head < 0) break;
            const int r = t * kTile + row;
            const int vis = p.causal ? min(it.keys, it.vis0 + r) : it.keys;
            const int j0 = it.j0, j_end = min(it.j1, it.n[t]);
            float m = -INFINITY, l = 0.f;
            for (int j = j0; j < j_end; ++j, ++s_uses) {
                ok = mla_wait(&sm->s_full[t], s_uses & 1, abort) && ok;
                __syncwarp();
                tc_fence_after();
                const int seen = vis - j * kTile - half * kHalf;  // of this thread's 64 keys
                uint32_t s[2][32];
                float2 sum[2];
                // Weights with the maximum of the steps before, which hardly ever has to be refreshed; at the first
                // step, and where some row's has grown too far, with one that is looked for first
                bool grown = true;
                for (bool look = j == j0;; look = true) {
                    tmem_ld32(s_at, s[0]);
                    tmem_ld32(s_at + 32, s[1]);
                    tmem_ld_wait();
                    if (seen < kHalf) {
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int y = 0; y < 32; ++y)
                                if (32 * x + y >= seen) s[x][y] = 0xFF800000u;
                    }
                    if (look) {
                        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int y = 0; y < 32; y += 2)
                                mx[x] = fmaxf(fmaxf(mx[x], __uint_as_float(s[x][y])), __uint_as_float(s[x][y + 1]));
                        sm->top[t][half][row] = grown ? fmaxf(mx[0], mx[1]) : -INFINITY;
                        bar_sync(two, 64);
                        const float top = fmaxf(sm->top[t][0][row], sm->top[t][1][row]);
                        if (j == j0) {
                            m = top;
                        } else if (__any_sync(0xffffffffu, top > m)) {
                            // Each row by its own scores: a neighbour's, which may be infinite, do not change its
                            // roundings.  QK of this step was issued behind PV of the one before, so O is at rest
                            const float fresh = fmaxf(top, m);
                            const float f = fresh == m ? 1.f : ex2_approx((m - fresh) * p.scale_log2);
                            m = fresh;
                            l *= f;
#pragma unroll 1
                            for (int x = 0; x < kHalf; x += 16) {
                                uint32_t o[16];
                                tmem_ld16(o_at + x, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                                tmem_st16(o_at + x, o);
                            }
                        }
                    }
                    const float nm = m == -INFINITY ? 0.f : -m * p.scale_log2;
                    const float2 nm2 = make_float2(nm, nm);
                    sum[0] = sum[1] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int y = 0; y < 16; ++y) {
                            const float a = __uint_as_float(s[x][2 * y]), b = __uint_as_float(s[x][2 * y + 1]);
                            float2 e = fma2(make_float2(a, b), c2, nm2);
                            e.x = ex2_approx(e.x);
                            e.y = ex2_approx(e.y);
                            sum[y & 1] = add2(sum[y & 1], e);
                            s[x][y] = pack_bf16(e.x, e.y);
                        }
                    sum[0] = add2(sum[0], sum[1]);
                    // Their sum says whether weights are too large; a row without a maximum needs one at its first scores.
                    // The row's two threads agree
                    grown = sum[0].x + sum[0].y > kGrown || (m == -INFINITY && seen > 0);
                    if (!bar_red_or(two, 64, grown) || look) break;
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t w[16];
#pragma unroll
                    for (int y = 0; y < 16; ++y) w[y] = s[x][y];
                    tmem_st16(s_at + 16 * x, w);
                }
                l += sum[0].x + sum[0].y;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->go[t]);
            }
            // ---- the query's result: its sum, then 64 of its values a thread.  What does not need the last
            // product comes before it
            const bool any = j0 < j_end, mine = r < it.rows;
            const int col = half * kHalf, masked = first_masked(it);
            if (any) {
                sm->top[t][half][row] = l;
                bar_sync(two, 64);
                l = sm->top[t][0][row] + sm->top[t][1][row];  // (written again behind the next item's first barrier)
            }
            const float lse = l > 0.f ? fmaf(m, p.scale, logf(l)) : l == l ? -INFINITY : l;
            const Place to = place(p, it, r, col, l > 0.f ? 1.f / l : l == l ? 0.f : l);
            float *lse_at = (it.joined ? p.part_lse + (int64_t)it.part * p.total_q * p.H : p.lse) + (it.row0 + r) * p.H + it.head;
            if (mine && half == 0 && it.part == 0)  // the join sees nothing in parts that this request does not have
                for (int x = it.parts; x < it.joined; ++x) lse_at[(int64_t)x * p.total_q * p.H] = -INFINITY;
            uint32_t o[2][32];  // (without a step whatever is there: l is 0 then)
            bool again = false;
            // (the last `go` is over then, and behind it what the scanning warps wrote of this tile's steps)
            if (any) ok = mla_wait(&sm->o_full[t], o_uses++ & 1, abort) && mla_wait(&sm->go[t], (s_uses - 1) & 1, abort) && ok;
            __syncwarp();
            tc_fence_after();
            tmem_ld32(o_at, o[0]);
            tmem_ld32(o_at + 32, o[1]);
            tmem_ld_wait();
            if (any && j_end > masked && !it.careful) {
                // A value that is not finite, at a key of a masked step, reaches queries that do not see it (as
                // 0 x inf).  That shows in the result; then the item is done again, with such values taken out
                float2 z[4] = {};
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    z[x % 4] = fma2(make_float2(__uint_as_float(o[x / 16][x % 16 * 2]), __uint_as_float(o[x / 16][x % 16 * 2 + 1])),
                                    make_float2(0.f, 0.f), z[x % 4]);
                z[0] = add2(add2(z[0], z[1]), add2(z[2], z[3]));
                again = bar_red_or(two, 64, mine && !(z[0].x + z[0].y == 0.f));
            }
            const bool odd = it.careful && sm->odd[i & 1];
            tc_fence_before();
            if (again) {
                if (lane == 0) sm->again[i & 1] = 1;
                item_done(i);
                continue;
            }
            if (odd && any) {
                rows_with_odd(p, it, r, min(vis, j_end * kTile), max(masked, j0) * kTile, min(j_end * kTile, it.keys), l, col, o_at);
                tc_fence_before();
                item_done(i);
            } else {
                item_done(i);  // before the stores, whose end it would otherwise wait for
                if (l == 0.f) {  // no weight at all, or nothing to weigh: 0, and not 0 x NaN
#pragma unroll
                    for (int x = 0; x < 64; ++x) o[x / 32][x % 32] = 0u;
                }
                if (mine) {
                    store32(to, 0, o[0]);
                    store32(to, 1, o[1]);
                }
            }
            if (mine && half == 0) *lse_at = lse;
            __syncwarp();
        }
        if (!ok && lane == 0) set_status(p.status, NSA_ERR_TIMEOUT);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) {
        tmem_relinquish();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Blocks of 256 queries that B requests of total_q queries have at most.
int64_t most_blocks(int B, int total_q)
{
    const int64_t n = ((int64_t)total_q + (int64_t)(kBlock - 1) * B) / kBlock;
    return n < total_q ? n : total_q;
}

// Parts are for calls of fewer items an SM than this, which bounds the workspace.
constexpr int kPartItems = 4;
constexpr size_t kHeadBytes = 256;  // of the workspace, before the parts: the items taken, the parts made

int most_parts_of(int B, int total_q, int total_k, int H, bool causal, int sms)
{
    const int64_t items = ceil_div(total_q, kBlock) * H;  // at least
    if (items >= (int64_t)kPartItems * sms || total_k <= 2 * kTile) return 1;
    const int64_t fit = (int64_t)kPartItems * sms * kBlock / ((int64_t)total_q * H);
    const int most = (int)(fit < 1 ? 1 : fit < kMaxMergeParts ? fit : kMaxMergeParts);
    if (B > 1) return most;  // the device knows the lengths
    const int blocks = ceil_of(total_q, kBlock), longest = block_steps(total_q, total_k, causal, blocks - 1);
    int64_t steps = 0;
    for (int i = 0; i < blocks; ++i) steps += block_steps(total_q, total_k, causal, i);
    int best = 1;
    float cost = parts_cost((float)items, longest, (float)(steps * H), 0.f, (float)sms);
    for (int c = 2; c <= most && c <= longest; ++c) {
        const int share = ceil_of(longest, c);
        const float x = parts_cost((float)items * c, share, (float)(steps * H), (float)total_q * H * c, (float)sms);
        if (x < cost) {
            cost = x;
            best = c;
        }
    }
    return best;
}

// Heads of a section (decode): as many as leave their keys and values (512 bytes a key) in L2, but enough for
// kSectionItems items an SM, since a section's items end with the short ones, which even the SMs out; and sections of
// one size, so that the last one is no rest of a few long items.
constexpr int64_t kL2Keys = 40LL << 20;
constexpr int kSectionItems = 4;

int heads_at_once_of(int64_t blocks, int total_k, int H, int sms)
{
    const int64_t fit = kL2Keys / ((int64_t)(total_k > 0 ? total_k : 1) * 2 * (kMlaNope + kMlaV));
    const int64_t fill = ceil_div((int64_t)kSectionItems * sms, blocks);
    const int64_t most = fit > fill ? fit : fill;
    return most >= H ? H : (int)ceil_div(H, ceil_div(H, most));
}

}  // namespace
}  // namespace nsa

extern "C" size_t nsa_mla_prefill_workspace_bytes(void)
{
    // most_parts_of: parts x queries x heads <= kPartItems x SMs x 256
    const int sms = nsa::current_sm_count();
    return nsa::kHeadBytes + (size_t)(sms > 0 ? sms : 0) * nsa::kPartItems * nsa::kBlock * (nsa::kMlaV + 1) * sizeof(float);
}

extern "C" nsa_status nsa_mla_prefill(const void *q_nope_dev, int64_t qn_ld_r, int64_t qn_ld_h, const void *q_rope_dev,
                                      int64_t qr_ld_r, int64_t qr_ld_h, const void *k_nope_dev, int64_t kn_ld_r,
                                      int64_t kn_ld_h, const void *k_rope_dev, int64_t kr_ld_r, const void *v_dev,
                                      int64_t v_ld_r, int64_t v_ld_h, const int32_t *cu_seqlens_q_dev,
                                      const int32_t *cu_seqlens_k_dev, int B, int total_q, int total_k, int H, int d_nope,
                                      int d_rope, int d_v, int causal, float sm_scale, void *out_dev, float *lse_dev,
                                      void *workspace_dev, size_t workspace_bytes, int32_t *status_dev, nsa_stream_t stream)
{
    using namespace nsa;
    if (B < 0 || total_q < 0 || total_k < 0 || H < 1 || causal < 0 || causal > 1) return NSA_ERR_INVALID_ARG;
    if (!(sm_scale > 0.f) || !(sm_scale < INFINITY)) return NSA_ERR_INVALID_ARG;
    if (d_nope != kMlaNope || d_rope != kMlaRope || d_v != kMlaV || H > 65535 || total_k > (1 << 30) || total_q > (1 << 30))
        return NSA_ERR_UNSUPPORTED;
    if (B == 0 || total_q == 0) return NSA_OK;
    if (!q_nope_dev || !q_rope_dev || !cu_seqlens_q_dev || !cu_seqlens_k_dev || !out_dev || !lse_dev || !workspace_dev ||
        (total_k > 0 && (!k_nope_dev || !k_rope_dev || !v_dev)))
        return NSA_ERR_INVALID_ARG;
    const uintptr_t wide = (uintptr_t)q_nope_dev | (uintptr_t)q_rope_dev | (uintptr_t)k_nope_dev | (uintptr_t)k_rope_dev |
                           (uintptr_t)v_dev | (uintptr_t)out_dev | (uintptr_t)workspace_dev;
    const uintptr_t word = (uintptr_t)cu_seqlens_q_dev | (uintptr_t)cu_seqlens_k_dev | (uintptr_t)lse_dev | (uintptr_t)status_dev;
    if ((wide & 15) || (word & 3)) return NSA_ERR_INVALID_ARG;
    // [rows][heads][d] with strides that TMA can step over; a single row's or head's stride is arbitrary
    struct Strided { int64_t *r, *h; int rows, d; };
    Strided all[5] = {{&qn_ld_r, &qn_ld_h, total_q, kMlaNope}, {&qr_ld_r, &qr_ld_h, total_q, kMlaRope},
                      {&kn_ld_r, &kn_ld_h, total_k, kMlaNope}, {&kr_ld_r, nullptr, total_k, kMlaRope},
                      {&v_ld_r, &v_ld_h, total_k, kMlaV}};
    for (const Strided &x : all) {
        if (x.h && H == 1) *x.h = x.d;
        if (x.rows <= 1) *x.r = x.h ? *x.h * H : x.d;
        if (*x.r < x.d || (x.h && *x.h < x.d) || *x.r % 8 || (x.h && *x.h % 8)) return NSA_ERR_INVALID_ARG;
        if (*x.r >= ((int64_t)1 << 38) || (x.h && *x.h >= ((int64_t)1 << 38))) return NSA_ERR_UNSUPPORTED;
    }
    if (workspace_bytes < nsa_mla_prefill_workspace_bytes()) return NSA_ERR_INVALID_ARG;
    const int sms = current_sm_count();
    if (sms <= 0) return NSA_ERR_CUDA;

    Params p;
    p.cu_q = cu_seqlens_q_dev; p.cu_k = cu_seqlens_k_dev;
    p.B = B; p.total_q = total_q; p.total_k = total_k; p.H = H; p.causal = causal;
    const int64_t items = most_blocks(B, total_q) * H;
    p.most_blocks = (int)most_blocks(B, total_q);
    p.most_parts = most_parts_of(B, total_q, total_k, H, causal, sms);
    p.heads_at_once = heads_at_once_of(p.most_blocks, total_k, H, sms);
    p.scale = sm_scale;
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    p.q_nope = (const __nv_bfloat16 *)q_nope_dev; p.q_rope = (const __nv_bfloat16 *)q_rope_dev;
    p.k_nope = (const __nv_bfloat16 *)k_nope_dev; p.k_rope = (const __nv_bfloat16 *)k_rope_dev;
    p.v = (const __nv_bfloat16 *)v_dev;
    p.qn_r = qn_ld_r; p.qn_h = qn_ld_h; p.qr_r = qr_ld_r; p.qr_h = qr_ld_h;
    p.kn_r = kn_ld_r; p.kn_h = kn_ld_h; p.kr_r = kr_ld_r; p.v_r = v_ld_r; p.v_h = v_ld_h;
    p.out = (__nv_bfloat16 *)out_dev; p.lse = lse_dev;
    p.part_out = (float *)((uint8_t *)workspace_dev + kHeadBytes);
    p.part_lse = p.part_out + (int64_t)p.most_parts * total_q * H * kMlaV;
    p.wide = (((uintptr_t)out_dev & 31) == 0 ? 1 : 0) | (((uintptr_t)p.part_out & 31) == 0 ? 2 : 0);
    p.parts_used = p.most_parts > 1 ? (int32_t *)workspace_dev + 16 : nullptr;
    p.status = status_dev;

    CUtensorMap qn, qr, kn, kr, v;
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    const uint64_t h = (uint64_t)H, tq = (uint64_t)total_q;
    // without a key no load is issued: the maps then describe the queries
    const bool keys = total_k > 0;
    const uint64_t tk = keys ? (uint64_t)total_k : tq;
    const bool mapped =
        make_tma_3d(&qn, bf, q_nope_dev, kMlaNope, h, tq, qn_ld_h * 2, qn_ld_r * 2, 64, 1, kTile, sw) &&
        make_tma_3d(&qr, bf, q_rope_dev, kMlaRope, h, tq, qr_ld_h * 2, qr_ld_r * 2, 64, 1, kTile, sw) &&
        (keys ? make_tma_3d(&kn, bf, k_nope_dev, kMlaNope, h, tk, kn_ld_h * 2, kn_ld_r * 2, 64, 1, kTile, sw) &&
                    make_tma_2d(&kr, bf, k_rope_dev, kMlaRope, tk, kr_ld_r * 2, 64, kTile, sw) &&
                    make_tma_3d(&v, bf, v_dev, kMlaV, h, tk, v_ld_h * 2, v_ld_r * 2, 64, 1, kTile / 2, sw)
              : make_tma_3d(&kn, bf, q_nope_dev, kMlaNope, h, tk, qn_ld_h * 2, qn_ld_r * 2, 64, 1, kTile, sw) &&
                    make_tma_2d(&kr, bf, q_rope_dev, kMlaRope, tk, qr_ld_r * 2, 64, kTile, sw) &&
                    make_tma_3d(&v, bf, q_nope_dev, kMlaNope, h, tk, qn_ld_h * 2, qn_ld_r * 2, 64, 1, kTile / 2, sw));
    if (!mapped) return NSA_ERR_CUDA;
    NSA_CUDA_TRY(max_dynamic_smem<mla_prefill_kernel>((int)kSmem));
    const cudaStream_t s = (cudaStream_t)stream;
    const int64_t work = items * p.most_parts;
    if (work > 2147483647LL - 65536) return NSA_ERR_UNSUPPORTED;
    p.next = nullptr;
    if (work > sms) {
        p.next = (int *)workspace_dev;
        NSA_CUDA_TRY(cudaMemsetAsync(p.next, 0, sizeof(*p.next), s));
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(work < sms ? work : sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    NSA_CUDA_TRY(cudaLaunchKernelEx(&cfg, mla_prefill_kernel, qn, qr, kn, kr, v, p));
    if (p.most_parts == 1) return NSA_OK;
    MergeParts parts = {};
    for (int i = 0; i < p.most_parts; ++i) {
        parts.out[i] = p.part_out + (int64_t)i * total_q * H * kMlaV;
        parts.lse[i] = p.part_lse + (int64_t)i * total_q * H;
    }
    parts.live_from = cu_seqlens_q_dev;
    parts.live_to = cu_seqlens_q_dev + B;
    parts.live_rows = H;
    parts.used = p.parts_used;
    return merge_launch(NSA_DT_F32, NSA_DT_BF16, p.most_parts, parts, (int64_t)total_q * H, kMlaV, out_dev, lse_dev, s);
}
