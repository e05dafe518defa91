// msda_cache_tc_f16_int8.cu -- tensor-core attention of f16 queries over a cache of int8 codes.
#include "msda_cache_tc_kernel.cuh"

namespace msda {
template cudaError_t launch_cache_tc<false, kCacheInt8>(const CacheArgs&, int, int, cudaStream_t);
}  // namespace msda
