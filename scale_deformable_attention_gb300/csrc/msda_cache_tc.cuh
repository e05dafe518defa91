// msda_cache_tc.cuh -- launch of the tensor-core attention over the paged cache.
#pragma once

#include "msda_cache.cuh"

namespace msda {

// a.tile_rows: `nq` (1 or 2) row tiles of G heads of as many tokens as 128 rows hold; a.tile_keys and a.tail_keys: 128.
template <bool BF16, int F>
cudaError_t launch_cache_tc(const CacheArgs& a, int nq, int grid, cudaStream_t st);

}  // namespace msda
