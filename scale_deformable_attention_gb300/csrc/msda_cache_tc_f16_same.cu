// msda_cache_tc_f16_same.cu -- tensor-core attention of f16 queries over a cache of the same type.
#include "msda_cache_tc_kernel.cuh"

namespace msda {
template cudaError_t launch_cache_tc<false, kCacheSame>(const CacheArgs&, int, int, cudaStream_t);
}  // namespace msda
