// msda_attention_simt_f16.cu -- attention on the FMA pipe, f16 tensors.
#define MSDA_ATTENTION_SIMT_INSTANTIATE
#include "msda_attention_simt.cuh"

namespace msda {
MSDA_SIMT_INSTANCES(__half)
}  // namespace msda
