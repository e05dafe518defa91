// msda_attention_tc.cuh -- what the tensor-core attention kernels share:
// arguments, tile geometry, masks of a tile's pairs as bits, the warp that
// clears rows which take no part.
#pragma once

#include "msda_attention.cuh"
#include "msda_tcgen05.cuh"

namespace msda {

constexpr int kTcRows = 128;            // rows and keys a tile
constexpr uint32_t kTcTile = 128 * 128; // bytes of 128 rows of 64 channels

struct TcArgs {
    AttentionArgs a;
    int G, qpt, rows;     // heads side by side in a row tile, queries a tile, rows used (G * qpt)
    int qblocks;          // row blocks of a key head (forward), row tiles of a head (backward)
    const uint32_t* bits_t;  // the mask's bits with keys as rows: [Bm, Mm, S, Wq], or null
    long long bits_t_sb, bits_t_sh;
    int Wq;
    // Where the mask leaves anything, in tiles of 128 (null without a mask): for a tile of queries the first and last
    // tile of keys, for one of keys those of queries, as kTcFar - first and last + 1 (0: none): [Bm, Mm, tiles][2].
    const int2 *ext_q, *ext_k;
    long long ext_sb, ext_sh;  // batch and head, in rows of tiles
    int fix_rows;         // backward: rows without keys may occur, and are cleared
    float* delta_out;      // backward: -delta, which the query kernel works out itself where one tile holds all keys of its rows
    const float* scale_in; // f16: the largest squared norms (see attention_amax), else null
};

// Largest query-to-key limit: query q sees keys j < tc_seen(q).
__device__ __forceinline__ int tc_seen(const AttentionArgs& a, int q) {
    if (!a.causal) return a.S;
    const long long n = (long long)q + 1 + (a.S - a.Q);
    return n < 0 ? 0 : n < a.S ? (int)n : a.S;
}

constexpr int kTcFar = 1 << 30;

// Narrows the tiles [*t0, *t1) to those between the first and the last that the mask leaves anything of, for the tiles
// x0..x1 (of `tiles`) of the other axis and `heads` heads from h on.
__device__ __forceinline__ void tc_narrow(const TcArgs& p, const int2* ext, int tiles, int b, int h, int heads, int x0, int x1,
                                          int* t0, int* t1) {
    if (!ext) return;
    int first = 0, last = 0;
    if (p.ext_sh == 0) heads = 1;
    for (int i = 0; i < heads; ++i)
        for (int x = x0; x <= x1; ++x) {
            const int2 e = ext[(b * p.ext_sb + (h + i) * p.ext_sh) * tiles + x];
            first = max(first, e.x), last = max(last, e.y);
        }
    *t0 = max(*t0, kTcFar - first);
    *t1 = min(*t1, last);
}

// the lowest n bits, n clamped to 0..32
__device__ __forceinline__ uint32_t tc_low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// First and last + 1 key tile of [t0, t1) that hold a key which `km` leaves
// (all threads of the block; they see the same bytes).
__device__ __forceinline__ void tc_trim(const uint8_t* km, int S, int* t0, int* t1) {
    while (*t0 < *t1) {
        const int lo = *t0 * kTcRows;
        bool any = false;
        const int n = min(S, *t1 * kTcRows) - lo;
        // one tile at a time until one holds a key: padding lies at the end as a rule
        any = (int)threadIdx.x < min(n, kTcRows) && km[lo + threadIdx.x] != 0;
        if (__syncthreads_or(any)) break;
        ++*t0;
    }
    while (*t0 < *t1) {
        // 8 tiles at a time from the end
        const int hi = min(S, *t1 * kTcRows), lo = max(*t0, *t1 - 8) * kTcRows;
        bool any = false;
        for (int j = lo + threadIdx.x; j < hi; j += blockDim.x) any |= km[j] != 0;
        if (__syncthreads_or(any)) break;
        *t1 = max(*t0, *t1 - 8);
    }
    while (*t0 < *t1) {
        const int hi = min(S, *t1 * kTcRows), lo = (*t1 - 1) * kTcRows;
        const bool any = (int)threadIdx.x < hi - lo && km[lo + threadIdx.x] != 0;
        if (__syncthreads_or(any)) break;
        --*t1;
    }
}

// Clears the rows of a tile (NC blocks of 128 rows of 128 bytes) whose bit in
// w[4] is 0: one warp, eight lanes a row.  A cleared row gives scores of 0 and
// products of 0 whatever it held.
template <int NC>
__device__ __forceinline__ void tc_clear_rows(unsigned char* tile, const uint32_t (&w)[4], int lane) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (w[k] == 0xffffffffu) continue;
        for (int r = lane >> 3; r < 32; r += 4) {
            if ((w[k] >> r) & 1u) continue;
#pragma unroll
            for (int c = 0; c < NC; ++c)
                *reinterpret_cast<uint4*>(tile + c * kTcTile + (k * 32 + r) * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
    }
}

// Bits of 128 keys from `km` (bytes; beyond `n` keys: 0), the same in all lanes.
__device__ __forceinline__ void tc_key_words(const uint8_t* km, int n, int lane, uint32_t (&w)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int j = k * 32 + lane;
        w[k] = __ballot_sync(0xffffffffu, j < n && km[j] != 0);
    }
}

}  // namespace msda
