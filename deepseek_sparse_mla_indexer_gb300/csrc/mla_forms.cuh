// Shared by the kernels of latent attention's two forms: the products with the key/value
// up-projection (mla_project.cu), the attention over expanded keys and values
// (mla_prefill.cu) and the join of attention over parts of the keys (merge_attention.cu).
#pragma once

#include "nsa_internal.cuh"
#include "sm100_paged.cuh"
#include "tma_host.h"

namespace nsa {

constexpr int kMlaLatent = 512, kMlaRope = 64, kMlaNope = 128, kMlaV = 128;
constexpr int kMlaHeadRows = kMlaNope + kMlaV;  // of the up-projection, per head

// Longest wait inside a kernel, in SM clocks (about a second); then it gives up (NSA_ERR_TIMEOUT).
constexpr long long kMlaWait = 2000000000LL;

// Waits for a phase, at most `most` clocks, and no longer than until another warp of the block gave up.
__device__ __forceinline__ bool mla_wait(uint64_t *bar, uint32_t parity, volatile int *abort, long long most = kMlaWait)
{
    if (sm100::mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!sm100::mbar_try_wait(bar, parity)) {
        if (*abort || clock64() - t0 > most) {
            *abort = 1;
            return false;
        }
    }
    return true;
}

// Arrives on the barrier at this offset in CTA `rank` of the cluster, as word that tensor-core or TMA operations are
// done: no thread's own writes go with it, so it and its wait keep to the scope of a CTA (with the cluster's,
// each of them orders all memory and takes as long as a product of 256 x 256 x 64).
__device__ __forceinline__ void mbar_tell(uint64_t *bar, uint32_t rank)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(sm100::dsmem_addr(bar, rank)) : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A tile from shared memory to a 3D tensor; what lies outside the tensor is left out.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, int x, int y, int z, const void *src)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
                 "r"(sm100::smem_u32(src)), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// Until at most one of the thread's committed bulk stores has still to read its source.
__device__ __forceinline__ void bulk_wait_read_1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }

// Joins `n` parts ([rows, D] values, [rows] lse) into out and lse, as nsa_merge_attention does.
constexpr int kMaxMergeParts = 8;
struct MergeParts {
    const void *out[kMaxMergeParts];
    const float *lse[kMaxMergeParts];
    // Or, for what the launch before this one leaves (fp32 parts, a bf16 result), on the device: how many of the
    // parts there are (nothing is written if there is one), and of the rows only those from *live_from x live_rows
    // up to *live_to x live_rows are.  NULL: all
    const int32_t *used, *live_from, *live_to;
    int live_rows;
};
nsa_status merge_launch(nsa_dtype part_dtype, nsa_dtype out_dtype, int n, const MergeParts &parts, int64_t rows, int D,
                        void *out, float *lse, cudaStream_t stream);

}  // namespace nsa
