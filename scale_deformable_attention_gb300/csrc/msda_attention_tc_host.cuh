// msda_attention_tc_host.cuh -- launches of the tensor-core attention kernels.
#pragma once

#include "msda_attention_tc.cuh"

namespace msda {

// Row tiles of the forward a block takes: two where that leaves a block for
// each SM, else one.
cudaError_t launch_attention_tc_forward(const TcArgs& p, bool bf16, int nq, const CUtensorMap& q, const CUtensorMap& k,
                                        const CUtensorMap& v, cudaStream_t st);

// Backward: q and g (the output's gradient) as heads of 128 rows, k and v as key heads of 128 rows.
cudaError_t launch_attention_tc_grad_key(const TcArgs& p, bool bf16, const CUtensorMap& q, const CUtensorMap& k,
                                         const CUtensorMap& v, const CUtensorMap& g, cudaStream_t st);
cudaError_t launch_attention_tc_grad_query(const TcArgs& p, bool bf16, const CUtensorMap& q, const CUtensorMap& k,
                                           const CUtensorMap& v, const CUtensorMap& g, cudaStream_t st);
// f16: largest squared norms of the rows of dout (a.row_l2 set) and of v, into top[2] (cleared before)
cudaError_t launch_attention_amax(const AttentionArgs& a, const AttentionRows& rw, float* top, cudaStream_t st);

}  // namespace msda
