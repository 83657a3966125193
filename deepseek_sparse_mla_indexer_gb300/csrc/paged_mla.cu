// nsa_paged_mla: MLA attention of each request's newest token(s) over its
// whole paged latent cache.
//
// Row r (request b = r / rows_per_req) sees the positions s < row_len[r] of
// its request, kept at slot page_table[b, s / page_size] * page_size +
// s % page_size.  Keys and values share the latent (absorbed MLA, as in
// [DSA] _forward_flashmla_kv): per head h
//   x_s = sm_scale (q_nope . K_s[0:d_latent] + q_rope . K_s[d_latent:])
//   lse = ln sum_s exp(x_s)        out = sum_s exp(x_s - lse) K_s[0:d_latent]
//
// This file holds the entry points and the CUDA-core kernel for any dims, any
// page size and fp32; the tensor-core kernel of the 512 + 64 shape is in
// paged_mla_tc.cu.
#include "paged_mla.cuh"
#include "paged_mla_tc.cuh"

namespace nsa {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 32;    // keys per tile (one per lane in the softmax)
constexpr int kMaxAcc = 32;  // accumulator entries per thread: heads per block * d_latent <= 8192
constexpr int kMaxSmem = kPagedSimtSmem;  // dynamic; the kernel is allowed all of it, whatever a call needs

constexpr int64_t smem_of(int heads, int dq)
{
    return (int64_t)sizeof(float) * ((heads + kTile) * (int64_t)(dq + 1) + heads * kTile + 3 * heads);
}
static_assert(smem_of(1, kPagedMaxRow) <= kMaxSmem && kPagedMaxRow <= kThreads * kMaxAcc, "one head fits");

// One CTA per (row, group of HG heads): a streaming softmax over tiles of 32
// keys held in shared memory as fp32.  Simple and exact in fp32; bound by
// shared-memory reads (every multiply-add takes an operand from there).
template <int QDT, int KDT>
__global__ void __launch_bounds__(kThreads)
paged_mla_simt_kernel(PagedMlaArgs p, int HG, void *out, float *lse)
{
    extern __shared__ float smem[];
    __shared__ int64_t slot[kTile];
    const int r = blockIdx.x, h0 = blockIdx.y * HG, hg = min(HG, p.H - h0);
    const int dq = p.d_latent + p.d_rope, ld = dq + 1;
    float *qs = smem;              // [HG][dq+1]
    float *ks = qs + HG * ld;      // [kTile][dq+1]
    float *S = ks + kTile * ld;    // [HG][kTile]
    float *alpha = S + HG * kTile, *m_run = alpha + HG, *l_run = m_run + HG;

    for (int i = threadIdx.x; i < hg * dq; i += kThreads) {
        const int h = i / dq, d = i - h * dq;
        qs[h * ld + d] = d < p.d_latent
                             ? load_elem<QDT>(p.q_nope, r * p.nope_ld_r + (int64_t)(h0 + h) * p.nope_ld_h + d)
                             : load_elem<QDT>(p.q_rope, r * p.rope_ld_r + (int64_t)(h0 + h) * p.rope_ld_h + d - p.d_latent);
    }
    for (int h = threadIdx.x; h < HG; h += kThreads) {
        m_run[h] = -INFINITY;
        l_run[h] = 0.f;
    }
    float acc[kMaxAcc];
    const int n_acc = (hg * p.d_latent + kThreads - 1) / kThreads;
#pragma unroll
    for (int i = 0; i < kMaxAcc; ++i) acc[i] = 0.f;

    const int L = checked_row_len(p.row_len, r, p.max_row_len, p.status);
    const int32_t *pt = p.page_table + (int64_t)(r / p.rows_per_req) * p.pt_ld;
    for (int j0 = 0; j0 < L; j0 += kTile) {
        __syncthreads();
        if (threadIdx.x < kTile)
            slot[threadIdx.x] =
                j0 + (int)threadIdx.x < L ? paged_slot(pt, j0 + threadIdx.x, p.page_size, p.num_pages, p.status) : -1;
        __syncthreads();
        for (int i = threadIdx.x; i < kTile * dq; i += kThreads) {
            const int j = i / dq, d = i - j * dq;
            ks[j * ld + d] = slot[j] >= 0 ? load_cache<KDT>(p.kv, slot[j], d, p.d_latent, p.d_rope) : 0.f;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < hg * kTile; e += kThreads) {
            const int h = e / kTile, j = e - h * kTile;
            float dot = 0.f;
            for (int d = 0; d < dq; ++d) dot = fmaf(qs[h * ld + d], ks[j * ld + d], dot);
            S[e] = slot[j] >= 0 ? dot * p.sm_scale : -INFINITY;
        }
        __syncthreads();
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        for (int h = warp; h < hg; h += kThreads / 32) {
            const float x = S[h * kTile + lane];
            float mx = x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float m_old = m_run[h], m_new = fmaxf(m_old, mx);
            const float pj = x == -INFINITY ? 0.f : expf(x - m_new);
            float sum = pj;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            S[h * kTile + lane] = pj;
            __syncwarp();
            if (lane == 0) {
                const float a = m_old == -INFINITY ? 0.f : expf(m_old - m_new);
                alpha[h] = a;
                m_run[h] = m_new;
                l_run[h] = l_run[h] * a + sum;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kMaxAcc; ++i) {
            const int e = threadIdx.x + i * kThreads;
            if (i < n_acc && e < hg * p.d_latent) {
                const int h = e / p.d_latent, d = e - h * p.d_latent;
                float v = acc[i] * alpha[h];
                for (int j = 0; j < kTile; ++j) v = fmaf(S[h * kTile + j], ks[j * ld + d], v);
                acc[i] = v;
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMaxAcc; ++i) {
        const int e = threadIdx.x + i * kThreads;
        if (i < n_acc && e < hg * p.d_latent) {
            const int h = e / p.d_latent, d = e - h * p.d_latent;
            // all scores -inf, or none: acc holds zeros, or the NaN of 0 x inf
            const float l = l_run[h], v = l > 0.f ? acc[i] / l : l == l ? acc[i] : l;
            const int64_t o = ((int64_t)r * p.H + h0 + h) * p.d_latent + d;
            if (QDT == NSA_DT_BF16)
                ((__nv_bfloat16 *)out)[o] = __float2bfloat16_rn(v);  // the result's type
            else
                ((float *)out)[o] = v;
        }
    }
    for (int h = threadIdx.x; h < hg; h += kThreads) {
        const float l = l_run[h];
        lse[(int64_t)r * p.H + h0 + h] = l > 0.f ? m_run[h] + logf(l) : l == l ? -INFINITY : l;
    }
}

template <int QDT, int KDT>
nsa_status launch_simt(const PagedMlaArgs &a, void *out, float *lse, cudaStream_t stream)
{
    // as many heads as the accumulators and shared memory hold: one at least (kPagedMaxRow)
    int HG = a.H < 16 ? a.H : 16;
    while (HG > 1 && (HG * a.d_latent > kThreads * kMaxAcc || smem_of(HG, a.d_latent + a.d_rope) > kMaxSmem)) --HG;
    const int64_t smem = smem_of(HG, a.d_latent + a.d_rope);
    constexpr auto k = paged_mla_simt_kernel<QDT, KDT>;
    NSA_CUDA_TRY(max_dynamic_smem<k>(kMaxSmem));
    k<<<dim3((unsigned)a.R, (unsigned)ceil_div(a.H, HG)), kThreads, (size_t)smem, stream>>>(a, HG, out, lse);
    return launch_status();
}

}  // namespace
}  // namespace nsa

extern "C" size_t nsa_paged_mla_workspace_bytes(nsa_dtype q_dtype, nsa_dtype kv_dtype, int R, int rows_per_req, int H,
                                                int d_latent, int d_rope, int max_row_len)
{
    return nsa::paged_mla_tc_workspace_bytes(q_dtype, kv_dtype, R, rows_per_req, H, d_latent, d_rope, max_row_len);
}

extern "C" nsa_status nsa_paged_mla(nsa_dtype q_dtype, nsa_dtype kv_dtype, const void *q_nope_dev, int64_t nope_ld_r,
                                    int64_t nope_ld_h, const void *q_rope_dev, int64_t rope_ld_r, int64_t rope_ld_h,
                                    const void *kv_dev, int64_t num_pages, int page_size,
                                    const int32_t *page_table_dev, int64_t pt_ld, const int32_t *row_len_dev, int R,
                                    int rows_per_req, int H, int d_latent, int d_rope, int max_row_len, float sm_scale,
                                    void *out_dev, float *lse_dev, void *workspace_dev, size_t workspace_bytes,
                                    int32_t *status_dev, nsa_stream_t stream)
{
    using namespace nsa;
    const PagedMlaArgs a = {q_dtype, kv_dtype, q_nope_dev, q_rope_dev, nope_ld_r, nope_ld_h, rope_ld_r, rope_ld_h,
                            kv_dev, num_pages, page_size, page_table_dev, pt_ld, row_len_dev, R, rows_per_req, H,
                            d_latent, d_rope, max_row_len, sm_scale, status_dev};
    const nsa_status ok = check_paged_mla(a);
    if (ok != NSA_OK || R == 0) return ok;
    if (!out_dev || !lse_dev || ((uintptr_t)lse_dev & 3) || ((uintptr_t)out_dev & (q_dtype == NSA_DT_F32 ? 3 : 1)))
        return NSA_ERR_INVALID_ARG;
    const size_t need =
        nsa_paged_mla_workspace_bytes(q_dtype, kv_dtype, R, rows_per_req, H, d_latent, d_rope, max_row_len);
    if (need > 0 && (workspace_bytes < need || !workspace_dev || ((uintptr_t)workspace_dev & 15)))
        return NSA_ERR_INVALID_ARG;
    const cudaStream_t s = (cudaStream_t)stream;
    const nsa_status st = paged_mla_tc_try_launch(a, out_dev, lse_dev, workspace_dev, workspace_bytes, s);
    if (st != NSA_ERR_UNSUPPORTED) return st;
    if (q_dtype == NSA_DT_F32) return launch_simt<NSA_DT_F32, NSA_DT_F32>(a, out_dev, lse_dev, s);
    if (kv_dtype == NSA_DT_BF16) return launch_simt<NSA_DT_BF16, NSA_DT_BF16>(a, out_dev, lse_dev, s);
    return launch_simt<NSA_DT_BF16, NSA_DT_E4M3>(a, out_dev, lse_dev, s);
}
