// msda_rotary_f32.cu -- rotary kernels for f32 rows.
#define MSDA_ROTARY_INSTANTIATE
#include "msda_rotary.cuh"

namespace msda {
MSDA_ROTARY_INSTANCES(float)
}  // namespace msda
