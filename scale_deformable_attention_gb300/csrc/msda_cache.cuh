// msda_cache.cuh -- what the kernels of the paged cache share: arguments, the
// codes that a quantised cache holds, the plan that cuts ragged sequences into
// equal shares of work.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "msda_attention.cuh"

namespace msda {

constexpr int kCacheSame = 0, kCacheE4m3 = 1, kCacheInt8 = 2;
constexpr unsigned kCacheBad = 8u;  // device error bit: a length, count, page or index outside its range

// The cache: pages of `page` tokens (a power of two, 16 or more), sequence b's
// token i in page table[b, i / page].
struct CachePages {
    void *k, *v;
    uint8_t *ks, *vs;                                 // a byte a token and head, or null: scale 2^(byte - 127)
    long long k_sp, k_st, k_sh, v_sp, v_st, v_sh;     // strides in elements: page, token, head
    long long ks_sp, ks_st, ks_sh, vs_sp, vs_st, vs_sh;
    const int* table;
    long long table_sb;
    int pages, page, page_log2, longest;              // longest: tokens a sequence has at most
    unsigned* err;
};

struct CacheArgs {
    CachePages c;
    const int *lengths, *counts;                      // [B]; counts or null: all T
    const void *q, *nk, *nv;                          // queries; keys and values of the new tokens or null
    long long q_sb, q_st, q_sh, nk_sb, nk_st, nk_sh, nv_sb, nv_st, nv_sh;
    const uint8_t* mask;                              // [B|1, T, T] or null: new tokens in order
    long long mk_sb, mk_sq;
    int B, T, M, N, D, G;                             // G = M / N query heads share a key head
    int rows, row_tiles, tile_rows;                   // T * G rows a key head, cut into tiles of tile_rows
    int tile_keys, tail_keys;                         // keys a tile of work: of the cache, of the new tokens
    float c2;                                         // scale * log2(e)
    void* out;                                        // [B, T, M, D]
    float* lse;                                       // [B, M, T]
    float *part_o, *part_l2;                          // [2 a block][tile_rows][D], [2 a block][tile_rows]
    int2* units;                                      // of each unit: slot of its first part (-1: it has none), parts
    int blocks, least;                                // blocks of the grid; tiles a block takes at least
    int whole;                                        // a block a unit, nothing to join
};

__device__ __forceinline__ int cache_length(const CachePages& c, const int* lengths, int b) {
    const int n = lengths[b];
    if (n >= 0 && n <= c.longest) return n;
    atomicOr(c.err, kCacheBad);
    return n < 0 ? 0 : c.longest;
}
__device__ __forceinline__ int cache_count(const CachePages& c, const int* counts, int b, int T) {
    const int n = counts ? counts[b] : T;
    if (n >= 0 && n <= T) return n;
    atomicOr(c.err, kCacheBad);
    return n < 0 ? 0 : T;
}
// page number of a sequence's token, -1 (and the error bit) where the table holds none
__device__ __forceinline__ int cache_page(const CachePages& c, int b, int token) {
    const int p = c.table[b * c.table_sb + (token >> c.page_log2)];
    if ((unsigned)p < (unsigned)c.pages) return p;
    atomicOr(c.err, kCacheBad);
    return -1;
}

// ---- the plan ----
// A unit is a tile of rows of one key head of one sequence; its work are the
// tiles of keys that the rows see, one at least (rows that see nothing are
// written too).  All units' tiles stand in one line (sequence, head, row tile),
// which the blocks share out evenly: a block may end one unit and begin another,
// so the lengths of the sequences need no balance, and a unit that several blocks
// share is joined from their parts.  Any block finds its share from the lengths
// alone, which every warp adds up by itself.
struct CacheUnit {
    int b, n, rt;
    int length, count;   // of sequence b
    int cache_tiles, tiles;
};

__device__ __forceinline__ int cache_tail_keys(const CacheArgs& a, int rt, int count) {
    if (!a.nk) return 0;
    const int first = rt * a.tile_rows / a.G;
    if (first >= count) return 0;
    if (a.mask) return count;
    return min(count, (min(a.rows, (rt + 1) * a.tile_rows) - 1) / a.G + 1);
}
__device__ __forceinline__ void cache_unit_tiles(const CacheArgs& a, CacheUnit& u) {
    const bool any = u.rt * a.tile_rows / a.G < u.count;
    u.cache_tiles = any ? (u.length + a.tile_keys - 1) / a.tile_keys : 0;
    u.tiles = max(1, u.cache_tiles + (cache_tail_keys(a, u.rt, u.count) + a.tail_keys - 1) / a.tail_keys);
}
// tiles of all row tiles of one key head of sequence b
__device__ __forceinline__ int cache_head_tiles(const CacheArgs& a, int b) {
    CacheUnit u;
    u.b = b, u.n = 0;
    u.length = cache_length(a.c, a.lengths, b), u.count = cache_count(a.c, a.counts, b, a.T);
    int sum = 0;
    for (u.rt = 0; u.rt < a.row_tiles; ++u.rt) {
        cache_unit_tiles(a, u);
        sum += u.tiles;
    }
    return sum;
}
__device__ __forceinline__ void cache_unit_at(const CacheArgs& a, int b, int n, int rt, CacheUnit& u) {
    u.b = b, u.n = n, u.rt = rt;
    u.length = cache_length(a.c, a.lengths, b), u.count = cache_count(a.c, a.counts, b, a.T);
    cache_unit_tiles(a, u);
}
__device__ __forceinline__ void cache_next_unit(const CacheArgs& a, CacheUnit& u) {
    if (++u.rt == a.row_tiles) {
        u.rt = 0;
        if (++u.n == a.N) {
            u.n = 0, ++u.b;
            if (u.b >= a.B) return;
            u.length = cache_length(a.c, a.lengths, u.b), u.count = cache_count(a.c, a.counts, u.b, a.T);
        }
    }
    cache_unit_tiles(a, u);
}

// Whole warp.  Tiles of all sequences.
__device__ __forceinline__ int cache_all_tiles(const CacheArgs& a) {
    const int lane = threadIdx.x & 31;
    int sum = 0;
    for (int i = lane; i < a.B; i += 32) sum += cache_head_tiles(a, i) * a.N;
    return __reduce_add_sync(0xffffffffu, sum);
}
__device__ __forceinline__ int cache_share(const CacheArgs& a, int all) { return max((all + a.blocks - 1) / a.blocks, a.least); }

// Whole warp.  The unit and the tile within it at place x of the line.
__device__ __forceinline__ void cache_find(const CacheArgs& a, int x, CacheUnit& u, int* tile) {
    const int lane = threadIdx.x & 31;
    int b = 0, head = 1;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int mine = b0 + lane < a.B ? cache_head_tiles(a, b0 + lane) : 0;
        int upto = mine * a.N;
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, upto, w);
            if (lane >= w) upto += o;
        }
        const unsigned behind = __ballot_sync(0xffffffffu, upto > x);
        if (behind) {
            const int l = __ffs(behind) - 1;
            b = b0 + l;
            head = __shfl_sync(0xffffffffu, mine, l);
            x -= __shfl_sync(0xffffffffu, upto, l) - head * a.N;
            break;
        }
        x -= __shfl_sync(0xffffffffu, upto, 31);
    }
    const int n = x / head;
    x -= n * head;
    cache_unit_at(a, b, n, 0, u);
    while (x >= u.tiles) {
        x -= u.tiles;
        ++u.rt;
        cache_unit_tiles(a, u);
    }
    *tile = x;
}

// The share of a block: calls f(unit, first tile, tiles, slot) for each unit that it has tiles of; `slot`: where the part
// goes, -1 where the block has the whole unit.
template <typename F>
__device__ __forceinline__ void cache_walk(const CacheArgs& a, F f) {
    CacheUnit u;
    if (a.whole) {
        int id = blockIdx.x;
        const int rt = id % a.row_tiles;
        id /= a.row_tiles;
        cache_unit_at(a, id / a.N, id % a.N, rt, u);
        f(u, 0, u.tiles, -1);
        return;
    }
    const int all = cache_all_tiles(a), share = cache_share(a, all);
    const long long at = (long long)blockIdx.x * share;
    if (at >= all) return;
    const int x0 = (int)at;
    int left = min(share, all - x0);
    int tile;
    cache_find(a, x0, u, &tile);
    bool first = true;
    while (left > 0) {
        const int n = min(u.tiles - tile, left);
        if (tile == 0 && threadIdx.x == 0)  // its first block says where its parts are
            a.units[(u.b * a.N + u.n) * a.row_tiles + u.rt] =
                make_int2(n == u.tiles ? -1 : 2 * (int)blockIdx.x + (first ? 0 : 1), 1 + (u.tiles - n + share - 1) / share);
        f(u, tile, n, n == u.tiles ? -1 : 2 * (int)blockIdx.x + (first ? 0 : 1));
        left -= n, tile = 0, first = false;
        if (left > 0) cache_next_unit(a, u);
    }
}

// ---- codes ----

__device__ __forceinline__ float cache_scale(uint32_t byte) { return __uint_as_float(byte << 23); }  // 255: infinite, and with codes of 0 NaN

// two codes (the low 16 bits) as f16, exactly
__device__ __forceinline__ uint32_t cache_e4m3_f16(uint32_t two) {
    uint32_t r;
    const uint16_t h = (uint16_t)two;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
    return r;
}
// four codes as f16: lo = codes 0 and 1, hi = 2 and 3
template <int F>
__device__ __forceinline__ void cache_four_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (F == kCacheE4m3) {
        lo = cache_e4m3_f16(w), hi = cache_e4m3_f16(w >> 16);
    } else {  // 0x6400 + u is 1024 + u in f16: u = code + 128
        const uint32_t u = w ^ 0x80808080u;
        const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off), y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
        lo = *reinterpret_cast<const uint32_t*>(&x), hi = *reinterpret_cast<const uint32_t*>(&y);
    }
}

// Joins the parts of units that several blocks shared; `early`: as a programmatic dependent of the kernel that makes them.
cudaError_t launch_cache_join(const CacheArgs& a, int dtype, bool early, cudaStream_t st);

// Attention of few rows a key head (tiles of 16 or 32): 128 threads, `bytes` of shared memory a block, `resident` blocks an SM.
struct CacheRowsShape {
    int tile_rows, tile_keys, tail_keys, resident;
};
template <typename T>
CacheRowsShape cache_rows_shape(int format, int D, int rows);
template <typename T>
cudaError_t launch_cache_rows(const CacheArgs& a, int format, int grid, cudaStream_t st);

}  // namespace msda
