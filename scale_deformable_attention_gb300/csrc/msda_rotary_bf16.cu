// msda_rotary_bf16.cu -- rotary kernels for bf16 rows.
#define MSDA_ROTARY_INSTANTIATE
#include "msda_rotary.cuh"

namespace msda {
MSDA_ROTARY_INSTANCES(__nv_bfloat16)
}  // namespace msda
