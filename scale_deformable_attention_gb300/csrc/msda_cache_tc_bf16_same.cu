// msda_cache_tc_bf16_same.cu -- tensor-core attention of bf16 queries over a cache of the same type.
#include "msda_cache_tc_kernel.cuh"

namespace msda {
template cudaError_t launch_cache_tc<true, kCacheSame>(const CacheArgs&, int, int, cudaStream_t);
}  // namespace msda
