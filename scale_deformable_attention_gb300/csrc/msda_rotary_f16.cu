// msda_rotary_f16.cu -- rotary kernels for f16 rows.
#define MSDA_ROTARY_INSTANTIATE
#include "msda_rotary.cuh"

namespace msda {
MSDA_ROTARY_INSTANCES(__half)
}  // namespace msda
