// msda_attention_simt_bf16.cu -- attention on the FMA pipe, bf16 tensors.
#define MSDA_ATTENTION_SIMT_INSTANTIATE
#include "msda_attention_simt.cuh"

namespace msda {
MSDA_SIMT_INSTANCES(__nv_bfloat16)
}  // namespace msda
