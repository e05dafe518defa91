// msda_cache_tc_f16_e4m3.cu -- tensor-core attention of f16 queries over a cache of e4m3 codes.
#include "msda_cache_tc_kernel.cuh"

namespace msda {
template cudaError_t launch_cache_tc<false, kCacheE4m3>(const CacheArgs&, int, int, cudaStream_t);
}  // namespace msda
