// msda_attention.cuh -- arguments that the attention kernels share, and the
// element-wise tests that say which (query, key) pairs take part.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace msda {

constexpr int kAttnMaxChannels = 128;

struct AttentionArgs {
    const void *q, *k, *v;
    long long q_sb, q_ss, q_sh, k_sb, k_ss, k_sh, v_sb, v_ss, v_sh;  // strides in elements: batch, row, head
    const uint8_t* key_mask;  // [B, S] (under a mask [B|1, N|1, S]) or null: 0 = the key takes no part
    long long km_sb, km_sh;
    const uint8_t* mask;  // [B|1, M|1, Q, S] or null: 0 = the pair takes no part
    long long mk_sb, mk_sh, mk_sq;
    const uint32_t* bits;  // the mask as bits [Bm, Mm, Q, W] (W words a row, a multiple of 4), or null
    long long bits_sb, bits_sh;
    int W;
    int B, Q, S, M, N, D;
    int G;        // M / N query heads share a key head
    int causal;   // query i sees keys up to i + S - Q
    float scale;  // natural units
    float c2;     // scale * log2(e)
    void* out;    // [B, Q, M, D]
    float* lse;   // [B, M, Q]
    // a long key axis split between blocks: partial rows, then joined
    float* part_o;    // [splits][B, M, Q][D] normalised rows
    float* part_lse;  // [splits][B, M, Q], log2 units
    int splits, tiles_per_split;
    // backward
    const void* dout;     // [B, Q, M, D]
    const float* row_l2;  // -lse * log2(e) of the kernels' rows (f16 on the tensor cores: + kHalfScale), -inf where a row takes no part
    const float* row_dl;  // -delta, delta = sum_d dout * out of the kernels' rows
    void *dq, *dk, *dv;   // [B, Q, M, D], [B, S, N, D], [B, S, N, D]
    unsigned* err;
    const unsigned* odd;  // binary32 on the tensor cores: where set those kernels return, else the FMA pipe's behind them; null: no such pair
};

// The backward's per-row statistics: tiles of `rt` rows of a head; a tile's l2
// and delta lie side by side: [B, heads, tiles][2][rt].
struct AttentionRows {
    int rt, tiles, heads;
};

// f16 on the tensor cores, backward: probabilities are held times 2^14, so that a
// share of 2^-28 of a row still has all its bits and one of 2^-39 some; f16 holds
// 65504, which leaves a factor of 4 for an lse that binary32 holds to 1 (above
// 2^24).  (The forward's scale is its own: a reference that follows the tiles.)
constexpr float kHalfScale = 14.f;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float attn_inf() { return __int_as_float(0x7f800000); }

}  // namespace msda
