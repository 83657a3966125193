// Tensor-core path of nsa_paged_mla (paged_mla_tc.cu).
#pragma once
#include "paged_mla.cuh"

namespace nsa {
// NSA_ERR_UNSUPPORTED: the shape is left to the CUDA-core kernel.
nsa_status paged_mla_tc_try_launch(const PagedMlaArgs &a, void *out, float *lse, void *workspace, size_t workspace_bytes,
                                   cudaStream_t stream);
size_t paged_mla_tc_workspace_bytes(nsa_dtype q_dtype, nsa_dtype kv_dtype, int R, int rows_per_req, int H, int d_latent,
                                    int d_rope, int max_row_len);
}  // namespace nsa
