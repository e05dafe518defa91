// msda_cache_rows_f32.cu -- attention over the paged cache of few rows a key head, queries in f32.
#include "msda_cache_rows.cuh"

namespace msda {
template CacheRowsShape cache_rows_shape<float>(int, int, int);
template cudaError_t launch_cache_rows<float>(const CacheArgs&, int, int, cudaStream_t);
}  // namespace msda
