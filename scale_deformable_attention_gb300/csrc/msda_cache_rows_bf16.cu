// msda_cache_rows_bf16.cu -- attention over the paged cache of few rows a key head, queries in bf16.
#include "msda_cache_rows.cuh"

namespace msda {
template CacheRowsShape cache_rows_shape<__nv_bfloat16>(int, int, int);
template cudaError_t launch_cache_rows<__nv_bfloat16>(const CacheArgs&, int, int, cudaStream_t);
}  // namespace msda
