// Shared by the operators that read a whole paged latent (MLA) cache:
// nsa_paged_mla (paged_mla.cu) and nsa_mla_key_weights (mla_key_weights.cu).
#pragma once

#include "nsa_internal.cuh"

namespace nsa {

// One call's queries, cache and row lengths, as the C entry points take them.
struct PagedMlaArgs {
    nsa_dtype q_dtype, kv_dtype;
    const void *q_nope, *q_rope;
    int64_t nope_ld_r, nope_ld_h, rope_ld_r, rope_ld_h;
    const void *kv;
    int64_t num_pages;
    int page_size;
    const int32_t *page_table;  // [R / rows_per_req][pt_ld]
    int64_t pt_ld;
    const int32_t *row_len;     // [R]
    int R, rows_per_req, H, d_latent, d_rope, max_row_len;
    float sm_scale;
    int32_t *status;
};

// The CUDA-core kernels hold 32 cache rows and at least one head's query in shared memory as fp32.
constexpr int kPagedSimtSmem = 226 * 1024;
constexpr int kPagedMaxRow = 1751;  // d_latent + d_rope

// Sizes that the kernels index with 32 bits.
inline bool paged_mla_sizes_ok(int R, int rows_per_req, int H, int max_row_len)
{
    return H <= 65535 && max_row_len <= (1 << 30) && (int64_t)rows_per_req * H <= (1 << 20) &&
           (int64_t)R * H <= 2147483647LL;
}

// Host-side checks that both entry points make.  NSA_OK also for R == 0.
inline nsa_status check_paged_mla(const PagedMlaArgs &a)
{
    if (a.R < 0 || a.rows_per_req < 1 || a.R % a.rows_per_req != 0 || a.H < 1 || a.d_latent < 1 || a.d_rope < 0 ||
        a.page_size < 1 || a.num_pages < 0 || a.max_row_len < 0 || a.pt_ld < 0)
        return NSA_ERR_INVALID_ARG;
    if (!(a.sm_scale > 0.f) || !(a.sm_scale < INFINITY)) return NSA_ERR_INVALID_ARG;
    if (a.pt_ld < ceil_div(a.max_row_len, a.page_size)) return NSA_ERR_INVALID_ARG;
    const bool combo_ok =
        (a.q_dtype == NSA_DT_F32 && a.kv_dtype == NSA_DT_F32) ||
        (a.q_dtype == NSA_DT_BF16 && (a.kv_dtype == NSA_DT_BF16 || a.kv_dtype == NSA_DT_E4M3));
    if (!combo_ok) return NSA_ERR_UNSUPPORTED;
    if (a.kv_dtype == NSA_DT_E4M3 && (a.d_latent % 128 != 0 || a.d_rope % 2 != 0)) return NSA_ERR_UNSUPPORTED;
    if ((int64_t)a.d_latent + a.d_rope > kPagedMaxRow) return NSA_ERR_UNSUPPORTED;
    if (!paged_mla_sizes_ok(a.R, a.rows_per_req, a.H, a.max_row_len) || a.page_size > (1 << 24) ||
        a.num_pages > 2147483647LL / a.page_size)
        return NSA_ERR_UNSUPPORTED;
    if (a.R == 0) return NSA_OK;
    if (!a.q_nope || (a.d_rope > 0 && !a.q_rope) || !a.kv || !a.row_len || (a.max_row_len > 0 && !a.page_table) ||
        a.num_pages < 1)
        return NSA_ERR_INVALID_ARG;
    const uintptr_t elem = a.q_dtype == NSA_DT_F32 ? 3 : 1;
    if (((uintptr_t)a.q_nope & elem) || ((uintptr_t)a.q_rope & elem)) return NSA_ERR_INVALID_ARG;
    if ((uintptr_t)a.kv & (a.kv_dtype == NSA_DT_BF16 ? 1 : 3)) return NSA_ERR_INVALID_ARG;
    if (((uintptr_t)a.page_table | (uintptr_t)a.row_len | (uintptr_t)a.status) & 3) return NSA_ERR_INVALID_ARG;
    return NSA_OK;
}

// Length of row r clipped to what the call allows; a length outside
// [0, max_row_len] is reported and the row sees no key.
__device__ __forceinline__ int checked_row_len(const int32_t *row_len, int r, int max_row_len, int32_t *status)
{
    const int L = row_len[r];
    if (L >= 0 && L <= max_row_len) return L;
    set_status(status, NSA_ERR_BOUNDS);
    return 0;
}

// Slot of position `pos` of a request, or -1 (reported) for a page outside the cache.
__device__ __forceinline__ int64_t paged_slot(const int32_t *pt_row, int pos, int page_size, int64_t num_pages,
                                              int32_t *status)
{
    const int pg = pos / page_size;
    const int32_t page = pt_row[pg];
    if (page < 0 || page >= num_pages) {
        set_status(status, NSA_ERR_BOUNDS);
        return -1;
    }
    return (int64_t)page * page_size + (pos - pg * page_size);
}

template <int DT>
__device__ __forceinline__ float load_elem(const void *p, int64_t i)
{
    if (DT == NSA_DT_BF16) return bf16_bits_to_float(((const uint16_t *)p)[i]);
    return ((const float *)p)[i];
}

// Element d of cache row `slot`.  An e4m3 row stands for the values that
// nsa_dequantize_kv_paged gives (code x scale rounded to fp32, then to bf16), so
// attending a quantised cache equals attending its dequantised copy.
template <int KDT>
__device__ __forceinline__ float load_cache(const void *kv, int64_t slot, int d, int d_latent, int d_rope)
{
    if (KDT != NSA_DT_E4M3) return load_elem<KDT>(kv, slot * (d_latent + d_rope) + d);
    const int nb = d_latent / 128;
    const uint8_t *row = (const uint8_t *)kv + slot * (int64_t)(d_latent + 4 * nb + 2 * d_rope);
    if (d < d_latent) {
        const float sc = *(const float *)(row + d_latent + 4 * (d / 128));
        return __bfloat162float(__float2bfloat16_rn(__fmul_rn(e4m3_to_float(row[d]), sc)));
    }
    return bf16_bits_to_float(*(const uint16_t *)(row + d_latent + 4 * nb + 2 * (d - d_latent)));
}

}  // namespace nsa
