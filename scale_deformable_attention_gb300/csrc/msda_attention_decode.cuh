// msda_attention_decode.cuh -- launch of the attention of a few rows.
#pragma once

#include "msda_attention.cuh"

namespace msda {

constexpr int kDecodeRows = 8;  // queries times heads of a key head (16 bits: one)

// a.tiles_per_split: keys a block takes
template <typename T>
cudaError_t launch_attention_decode(const AttentionArgs& a, cudaStream_t st);

}  // namespace msda
