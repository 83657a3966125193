// nsa_merge_attention: attention over parts of the keys joined by the parts' lse,
//   lse = ln sum_p exp(lse_p)      out = sum_p exp(lse_p - lse) out_p
// as the chunks of a long prefix, or the shares of a row's keys, leave it.
//
// Bound by memory: every part is read once and the result written once, 16 bytes and more a
// thread and part, all parts' loads in flight together (three bf16 parts of 8192 x 128 rows of 128:
// 178 us, 6.1 TB/s, 92 % of a copy; 213 us when the values waited for their lse).  A thread block holds whole rows, so that
// the result may take the place of a part: every lse is read before any is written.
#include "mla_forms.cuh"

namespace nsa {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;  // values a thread
constexpr int kJoinBlocks = 4;  // an SM

__device__ __forceinline__ void load8(const float *p, float (&v)[kVec])
{
    const float4 a = __ldcs((const float4 *)p), b = __ldcs((const float4 *)(p + 4));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[kVec])
{
    const uint4 w = __ldcs((const uint4 *)p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void store8(float *p, const float (&v)[kVec])
{
    *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]);
    *(float4 *)(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[kVec])
{
    *(uint4 *)p = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// units: threads a row (D / 8); a block has kThreads / units rows.  USED: as many parts as the device says, and each
// block more than one lot of rows (which costs the other form 3 %).
template <typename In, typename Out, int NP, bool USED>
__global__ void __launch_bounds__(kThreads)
merge_kernel(const MergeParts parts, int64_t rows, int units, Out *out, float *lse)
{
    pdl_wait();
    int n = NP;
    int64_t from = 0;
    if constexpr (USED) {
        n = *parts.used;
        if (n <= 1) return;
        from = (int64_t)*parts.live_from * parts.live_rows;
        rows = min(rows, (int64_t)*parts.live_to * parts.live_rows);
    }
    const int per = kThreads / units, r = threadIdx.x / units, u = threadIdx.x - r * units;
    for (int64_t row0 = (int64_t)blockIdx.x * per; row0 < rows; row0 += (int64_t)gridDim.x * per) {
        const int64_t row = row0 + r, at = (row * units + u) * kVec;
        const bool live = r < per && row >= from && row < rows;
        float l[NP], x[NP][kVec], o[kVec], top = -INFINITY, total = 0.f;
        if (live) {
#pragma unroll
            for (int i = 0; i < NP; ++i) l[i] = i < n ? parts.lse[i][row] : -INFINITY;
            // (read without a look at the lse, so that one latency covers both)
#pragma unroll
            for (int i = 0; i < NP; ++i)
                if (i < n) load8((const In *)parts.out[i] + at, x[i]);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                if (l[i] == -INFINITY) {  // a part that saw no key has weight 0, whatever its values are
#pragma unroll
                    for (int j = 0; j < kVec; ++j) x[i][j] = 0.f;
                }
                top = fmaxf(top, l[i]);
            }
            if (top == -INFINITY) top = 0.f;  // no key in any part, or NaN
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                l[i] = expf(l[i] - top);
                total += l[i];
            }
            const float inv = total > 0.f ? 1.f / total : total;  // 0 without a key, NaN stays
            // divided before the sum, which then stays within the values' range
#pragma unroll
            for (int i = 0; i < NP; ++i) l[i] *= inv;
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                o[j] = 0.f;
#pragma unroll
                for (int i = 0; i < NP; ++i) o[j] = fmaf(l[i], x[i][j], o[j]);
            }
        }
        __syncthreads();  // every lse of the block's rows is read
        if (live) {
            store8(out + at, o);
            if (u == 0) lse[row] = total == 0.f ? -INFINITY : top + logf(total);
        }
        if constexpr (!USED) break;
    }
}

template <typename In, typename Out, int NP, bool USED = false>
nsa_status launch(const MergeParts &parts, int64_t rows, int D, Out *out, float *lse, cudaStream_t stream)
{
    const int units = D / kVec;
    cudaLaunchConfig_t cfg = {};
    int64_t blocks = ceil_div(rows, kThreads / units);
    if (USED) {  // there may be nothing to join: no more blocks than find that out at once
        const int sms = current_sm_count();
        if (blocks > (int64_t)sms * kJoinBlocks) blocks = (int64_t)sms * kJoinBlocks;
    }
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    NSA_CUDA_TRY(cudaLaunchKernelEx(&cfg, merge_kernel<In, Out, NP, USED>, parts, rows, units, out, lse));
    return NSA_OK;
}

template <typename In, typename Out>
nsa_status launch_n(int n, const MergeParts &parts, int64_t rows, int D, void *out, float *lse, cudaStream_t s)
{
    Out *o = (Out *)out;
    switch (n) {
    case 1: return launch<In, Out, 1>(parts, rows, D, o, lse, s);
    case 2: return launch<In, Out, 2>(parts, rows, D, o, lse, s);
    case 3: return launch<In, Out, 3>(parts, rows, D, o, lse, s);
    case 4: return launch<In, Out, 4>(parts, rows, D, o, lse, s);
    case 5: return launch<In, Out, 5>(parts, rows, D, o, lse, s);
    case 6: return launch<In, Out, 6>(parts, rows, D, o, lse, s);
    case 7: return launch<In, Out, 7>(parts, rows, D, o, lse, s);
    default: return launch<In, Out, 8>(parts, rows, D, o, lse, s);
    }
}

}  // namespace

nsa_status merge_launch(nsa_dtype part_dtype, nsa_dtype out_dtype, int n, const MergeParts &parts, int64_t rows, int D,
                        void *out, float *lse, cudaStream_t s)
{
    if (parts.used)
        return launch<float, __nv_bfloat16, kMaxMergeParts, true>(parts, rows, D, (__nv_bfloat16 *)out, lse, s);
    if (part_dtype == NSA_DT_BF16) return launch_n<__nv_bfloat16, __nv_bfloat16>(n, parts, rows, D, out, lse, s);
    if (out_dtype == NSA_DT_BF16) return launch_n<float, __nv_bfloat16>(n, parts, rows, D, out, lse, s);
    return launch_n<float, float>(n, parts, rows, D, out, lse, s);
}

}  // namespace nsa

extern "C" nsa_status nsa_merge_attention(nsa_dtype part_dtype, nsa_dtype out_dtype, int n_parts,
                                          const void *const *parts_dev, const float *const *lses_dev, int64_t rows, int D,
                                          void *out_dev, float *lse_dev, nsa_stream_t stream)
{
    using namespace nsa;
    if (n_parts < 1 || rows < 0 || D < 1 || !parts_dev || !lses_dev) return NSA_ERR_INVALID_ARG;
    const bool types = (part_dtype == NSA_DT_BF16 && out_dtype == NSA_DT_BF16) ||
                       (part_dtype == NSA_DT_F32 && (out_dtype == NSA_DT_BF16 || out_dtype == NSA_DT_F32));
    if (!types || n_parts > kMaxMergeParts || D % kVec != 0 || D > kVec * kThreads) return NSA_ERR_UNSUPPORTED;
    if (ceil_div(rows, kThreads / (D / kVec)) > 2147483647LL) return NSA_ERR_UNSUPPORTED;
    if (rows == 0) return NSA_OK;
    MergeParts parts = {};
    uintptr_t wide = (uintptr_t)out_dev, word = (uintptr_t)lse_dev;
    if (!out_dev || !lse_dev) return NSA_ERR_INVALID_ARG;
    for (int i = 0; i < n_parts; ++i) {
        if (!parts_dev[i] || !lses_dev[i]) return NSA_ERR_INVALID_ARG;
        parts.out[i] = parts_dev[i];
        parts.lse[i] = lses_dev[i];
        wide |= (uintptr_t)parts_dev[i];
        word |= (uintptr_t)lses_dev[i];
    }
    if ((wide & 15) || (word & 3)) return NSA_ERR_INVALID_ARG;
    return merge_launch(part_dtype, out_dtype, n_parts, parts, rows, D, out_dev, lse_dev, (cudaStream_t)stream);
}
