// msda_attention_simt_f32.cu -- attention on the FMA pipe, f32 tensors.
#define MSDA_ATTENTION_SIMT_INSTANTIATE
#include "msda_attention_simt.cuh"

namespace msda {
MSDA_SIMT_INSTANCES(float)
}  // namespace msda
