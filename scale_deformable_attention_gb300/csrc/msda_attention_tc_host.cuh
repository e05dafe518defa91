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

}  // namespace msda
