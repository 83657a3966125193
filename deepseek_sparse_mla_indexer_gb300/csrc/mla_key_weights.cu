// nsa_mla_key_weights: the attention weight that each cached position of a
// request receives, summed over the request's rows and heads and added to a
// running total per position:
//   total[b, s] += sum_{rows r of b, s < row_len[r]} sum_h exp(x_{r,h,s} - lse[r, h])
//   x_{r,h,s} = sm_scale (q_nope[r,h] . K_s[0:d_latent] + q_rope[r,h] . K_s[d_latent:])
// lse is what nsa_paged_mla wrote for the same rows.  The weights are computed
// again from q and K rather than kept by the attention: a split attention
// knows its log-sum-exp only after the join, and the weights of 128 heads (512
// bytes a key and pass, written and read) cost about what reading the key
// again does.
//
// This file holds the entry point and the CUDA-core kernel for any dims; the
// tensor-core kernel of the 512 + 64 shape is in mla_key_weights_tc.cu.
#include "mla_key_weights_tc.cuh"

namespace nsa {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 32;  // keys per CTA, one per lane
constexpr int kHG = 16;    // heads staged at once, at most
constexpr int kMaxSmem = kPagedSimtSmem;  // dynamic; the kernel is allowed all of it, whatever a call needs

constexpr int64_t smem_of(int heads, int dq)
{
    return (int64_t)sizeof(float) * (kTile * (int64_t)(dq + 1) + (int64_t)heads * dq);
}
static_assert(smem_of(1, kPagedMaxRow) <= kMaxSmem, "one head fits");

// One CTA per (request, 32 keys).  Every warp takes every eighth head of each
// row; the warps' sums are joined in a fixed order, so the result does not
// depend on scheduling.
template <int QDT, int KDT>
__global__ void __launch_bounds__(kThreads) key_weights_simt_kernel(PagedMlaArgs p, int HG, const float *lse,
                                                                    float *total, int64_t total_ld)
{
    extern __shared__ float smem[];
    __shared__ int64_t slot[kTile];
    const int dq = p.d_latent + p.d_rope, ld = dq + 1;
    float *ks = smem, *qs = ks + kTile * ld;
    const int per = (p.max_row_len + kTile - 1) / kTile, b = blockIdx.x / per, j0 = (blockIdx.x - b * per) * kTile;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int longest = 0;
    for (int i = 0; i < p.rows_per_req; ++i)
        longest = max(longest, checked_row_len(p.row_len, b * p.rows_per_req + i, p.max_row_len, p.status));
    if (j0 >= longest) return;
    if (threadIdx.x < kTile)
        slot[threadIdx.x] = j0 + (int)threadIdx.x < longest
                                ? paged_slot(p.page_table + (int64_t)b * p.pt_ld, j0 + threadIdx.x, p.page_size,
                                             p.num_pages, p.status)
                                : -1;
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * dq; i += kThreads) {
        const int j = i / dq, d = i - j * dq;
        ks[j * ld + d] = slot[j] >= 0 ? load_cache<KDT>(p.kv, slot[j], d, p.d_latent, p.d_rope) : 0.f;
    }
    float sum = 0.f;
    for (int i = 0; i < p.rows_per_req; ++i) {
        const int64_t r = (int64_t)b * p.rows_per_req + i;
        const int L = p.row_len[r];
        if (L < 0 || L > p.max_row_len) continue;
        for (int h0 = 0; h0 < p.H; h0 += HG) {
            const int hg = min(HG, p.H - h0);
            __syncthreads();
            for (int e = threadIdx.x; e < hg * dq; e += kThreads) {
                const int h = e / dq, d = e - h * dq;
                qs[e] = d < p.d_latent
                            ? load_elem<QDT>(p.q_nope, r * p.nope_ld_r + (int64_t)(h0 + h) * p.nope_ld_h + d)
                            : load_elem<QDT>(p.q_rope, r * p.rope_ld_r + (int64_t)(h0 + h) * p.rope_ld_h + d - p.d_latent);
            }
            __syncthreads();
            for (int h = warp; h < hg; h += kThreads / 32) {
                float dot = 0.f;
                for (int d = 0; d < dq; ++d) dot = fmaf(qs[h * dq + d], ks[lane * ld + d], dot);
                const float ls = lse[r * p.H + h0 + h];
                // a row that saw no key (lse -inf) gives no weight
                if (j0 + lane < L && slot[lane] >= 0 && ls != -INFINITY) sum += expf(dot * p.sm_scale - ls);
            }
        }
    }
    float *part = smem;  // [warps][kTile], where the keys were
    __syncthreads();
    part[warp * kTile + lane] = sum;
    __syncthreads();
    if (threadIdx.x < kTile && slot[threadIdx.x] >= 0) {
        float w = 0.f;
        for (int k = 0; k < kThreads / 32; ++k) w += part[k * kTile + threadIdx.x];
        total[b * total_ld + j0 + threadIdx.x] += w;
    }
}

template <int QDT, int KDT>
nsa_status launch_simt(const PagedMlaArgs &a, const float *lse, float *total, int64_t total_ld, cudaStream_t stream)
{
    const int dq = a.d_latent + a.d_rope;
    int HG = a.H < kHG ? a.H : kHG;
    while (HG > 1 && smem_of(HG, dq) > kMaxSmem) --HG;
    const int64_t part = (int64_t)sizeof(float) * kThreads;
    const int64_t smem = smem_of(HG, dq) > part ? smem_of(HG, dq) : part;
    const int64_t blocks = ceil_div(a.max_row_len, kTile) * (a.R / a.rows_per_req);
    if (blocks > 2147483647LL) return NSA_ERR_UNSUPPORTED;
    constexpr auto k = key_weights_simt_kernel<QDT, KDT>;
    NSA_CUDA_TRY(max_dynamic_smem<k>(kMaxSmem));
    k<<<(unsigned)blocks, kThreads, (size_t)smem, stream>>>(a, HG, lse, total, total_ld);
    return launch_status();
}

}  // namespace
}  // namespace nsa

extern "C" nsa_status nsa_mla_key_weights(nsa_dtype q_dtype, nsa_dtype kv_dtype, const void *q_nope_dev,
                                          int64_t nope_ld_r, int64_t nope_ld_h, const void *q_rope_dev,
                                          int64_t rope_ld_r, int64_t rope_ld_h, const void *kv_dev, int64_t num_pages,
                                          int page_size, const int32_t *page_table_dev, int64_t pt_ld,
                                          const int32_t *row_len_dev, int R, int rows_per_req, int H, int d_latent,
                                          int d_rope, int max_row_len, float sm_scale, const float *lse_dev,
                                          float *total_dev, int64_t total_ld, int32_t *status_dev, nsa_stream_t stream)
{
    using namespace nsa;
    const PagedMlaArgs a = {q_dtype, kv_dtype, q_nope_dev, q_rope_dev, nope_ld_r, nope_ld_h, rope_ld_r, rope_ld_h,
                            kv_dev, num_pages, page_size, page_table_dev, pt_ld, row_len_dev, R, rows_per_req, H,
                            d_latent, d_rope, max_row_len, sm_scale, status_dev};
    const nsa_status ok = check_paged_mla(a);
    if (ok != NSA_OK || R == 0 || max_row_len == 0) return ok;
    if (!lse_dev || !total_dev || (((uintptr_t)lse_dev | (uintptr_t)total_dev) & 3) || total_ld < max_row_len)
        return NSA_ERR_INVALID_ARG;
    const cudaStream_t s = (cudaStream_t)stream;
    const nsa_status st = key_weights_tc_try_launch(a, lse_dev, total_dev, total_ld, s);
    if (st != NSA_ERR_UNSUPPORTED) return st;
    if (q_dtype == NSA_DT_F32) return launch_simt<NSA_DT_F32, NSA_DT_F32>(a, lse_dev, total_dev, total_ld, s);
    if (kv_dtype == NSA_DT_BF16) return launch_simt<NSA_DT_BF16, NSA_DT_BF16>(a, lse_dev, total_dev, total_ld, s);
    return launch_simt<NSA_DT_BF16, NSA_DT_E4M3>(a, lse_dev, total_dev, total_ld, s);
}
