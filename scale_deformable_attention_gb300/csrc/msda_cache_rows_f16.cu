// msda_cache_rows_f16.cu -- attention over the paged cache of few rows a key head, queries in f16.
#include "msda_cache_rows.cuh"

namespace msda {
template CacheRowsShape cache_rows_shape<__half>(int, int, int);
template cudaError_t launch_cache_rows<__half>(const CacheArgs&, int, int, cudaStream_t);
}  // namespace msda
