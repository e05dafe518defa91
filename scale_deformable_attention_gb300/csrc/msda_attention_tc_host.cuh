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

// binary32: tensors cut into three bf16 pieces [3][B, rows, heads, Dp]; rows that `alive` (bytes) or `lse` (-inf)
// leave out become zeros.
struct SplitTensor {
    const float* src;
    long long sb, ss, sh;  // strides in elements: batch, row, head
    long long rows;
    int heads;
    bool vec;              // rows of whole 16-byte vectors
    const uint8_t* alive;
    long long alive_sb, alive_sh;
    const float* lse;      // [B, heads, rows]
    void* dst;
};
struct SplitArgs {
    SplitTensor t[4];
    int B, D, Dp;
    unsigned* odd;  // set where a value is beyond 2^60, infinite or NaN
};
cudaError_t launch_attention_split(const SplitArgs& a, int tensors, cudaStream_t st);
cudaError_t launch_attention_tc_f32(const TcArgs& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                    cudaStream_t st);
cudaError_t launch_attention_tc_f32_grad_key(const TcArgs& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                             const CUtensorMap& g, cudaStream_t st);
cudaError_t launch_attention_tc_f32_grad_query(const TcArgs& p, const CUtensorMap& q, const CUtensorMap& k,
                                               const CUtensorMap& v, const CUtensorMap& g, cudaStream_t st);

}  // namespace msda
