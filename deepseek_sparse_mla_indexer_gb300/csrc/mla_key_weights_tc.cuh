// Tensor-core path of nsa_mla_key_weights (mla_key_weights_tc.cu).
#pragma once
#include "paged_mla.cuh"

namespace nsa {
// NSA_ERR_UNSUPPORTED: the shape is left to the CUDA-core kernel.
nsa_status key_weights_tc_try_launch(const PagedMlaArgs &a, const float *lse, float *total, int64_t total_ld,
                                     cudaStream_t stream);
}  // namespace nsa
