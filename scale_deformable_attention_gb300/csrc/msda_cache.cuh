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
    int tile_log2, tail_log2;                         // keys a tile of work: 2^tile_log2 of the cache, 2^tail_log2 of the new tokens
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
// The table's entry for a sequence's token, as it stands there: read ahead of its use, so that nothing waits for it.
constexpr int kCacheNoPage = -0x7fffffff;  // what a caller puts where there is no token; an entry of this value is no page either
__device__ __forceinline__ int cache_entry(const CachePages& c, int b, int token) { return c.table[b * c.table_sb + (token >> c.page_log2)]; }
// The page of an entry, -1 (and the error bit) where it is none.
__device__ __forceinline__ int cache_page_of(const CachePages& c, int entry) {
    if ((unsigned)entry < (unsigned)c.pages) return entry;
    if (entry != kCacheNoPage) atomicOr(c.err, kCacheBad);
    return -1;
}
__device__ __forceinline__ int cache_page(const CachePages& c, int b, int token) { return cache_page_of(c, cache_entry(c, b, token)); }

// ---- the plan ----
// A unit is a tile of rows of one key head of one sequence; its work are the
// tiles of keys that the rows see, one at least (rows that see nothing are
// written too).  All units' tiles stand in one line (sequence, head, row tile),
// which the blocks share out evenly: a block may end one unit and begin another,
// so the lengths of the sequences need no balance, and a unit that several blocks
// share is joined from their parts.  Any block finds its share from the lengths
// alone.
struct CacheUnit {
    int b, n, rt;
    int length, count;   // of sequence b
    int cache_tiles, tiles;
};

// new tokens that a row tile sees at most
__device__ __forceinline__ int cache_tail_keys(const CacheArgs& a, int rt, int count) {
    if (!a.nk) return 0;
    if (rt > 0 && rt * a.tile_rows / a.G >= count) return 0;
    if (a.mask || rt == a.row_tiles - 1) return count;
    return min(count, ((rt + 1) * a.tile_rows - 1) / a.G + 1);
}
__device__ __forceinline__ void cache_unit_tiles(const CacheArgs& a, CacheUnit& u) {
    const bool any = u.rt == 0 ? u.count > 0 : u.rt * a.tile_rows / a.G < u.count;
    u.cache_tiles = any ? (u.length + (1 << a.tile_log2) - 1) >> a.tile_log2 : 0;
    u.tiles = max(1, u.cache_tiles + ((cache_tail_keys(a, u.rt, u.count) + (1 << a.tail_log2) - 1) >> a.tail_log2));
}
// tiles of all row tiles of one key head of sequence b
__device__ __forceinline__ int cache_head_tiles(const CacheArgs& a, int b) {
    CacheUnit u;
    u.length = cache_length(a.c, a.lengths, b), u.count = cache_count(a.c, a.counts, b, a.T);
    int sum = 0;
#pragma unroll 1
    for (u.rt = 0; u.rt < a.row_tiles; ++u.rt) {
        cache_unit_tiles(a, u);
        sum += u.tiles;
    }
    return sum;
}
__device__ __forceinline__ void cache_next_unit(const CacheArgs& a, CacheUnit& u) {
    if (++u.rt == a.row_tiles) {
        u.rt = 0;
        if (++u.n == a.N) {
            u.n = 0, ++u.b;
            u.length = cache_length(a.c, a.lengths, u.b), u.count = cache_count(a.c, a.counts, u.b, a.T);
        }
    }
    cache_unit_tiles(a, u);
}

// Where a block begins: its first unit, the tile within it, its tiles in all and those of each block.  One warp works it out for
// its block (code that runs once costs about 9 cycles an instruction to fetch, and each role of a block would have its own).
struct CacheStart {
    CacheUnit u;
    int tile, left, share;
};

// Whole warp, all lanes with the same result.
__device__ __forceinline__ CacheStart cache_start(const CacheArgs& a) {
    const int lane = threadIdx.x & 31;
    CacheStart s;
    s.tile = s.left = s.share = 0;
    int rt = 0;
    if (a.whole) {
        const int id = blockIdx.x / a.row_tiles;
        rt = blockIdx.x - id * a.row_tiles;
        s.u.b = id / a.N, s.u.n = id - s.u.b * a.N;
    } else {
        int all = 0;
#pragma unroll 1
        for (int i = lane; i < a.B; i += 32) all += cache_head_tiles(a, i) * a.N;
        all = __reduce_add_sync(0xffffffffu, all);
        s.share = max((all + a.blocks - 1) / a.blocks, a.least);
        const long long at = (long long)blockIdx.x * s.share;
        if (at >= all) return s;
        int x = (int)at, head = 1;
        s.left = min(s.share, all - x);
        s.u.b = 0;
#pragma unroll 1
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
                s.u.b = b0 + l;
                head = __shfl_sync(0xffffffffu, mine, l);
                x -= __shfl_sync(0xffffffffu, upto, l) - head * a.N;
                break;
            }
            x -= __shfl_sync(0xffffffffu, upto, 31);
        }
        s.u.n = x / head;
        s.tile = x - s.u.n * head;
    }
    s.u.rt = rt;
    s.u.length = cache_length(a.c, a.lengths, s.u.b), s.u.count = cache_count(a.c, a.counts, s.u.b, a.T);
    cache_unit_tiles(a, s.u);
    if (a.whole) {
        s.left = s.share = s.u.tiles;
    } else {
#pragma unroll 1
        while (s.tile >= s.u.tiles) {
            s.tile -= s.u.tiles;
            ++s.u.rt;
            cache_unit_tiles(a, s.u);
        }
    }
    return s;
}

// The share of a block: calls f(unit, first tile, tiles, slot) for each unit that it has tiles of; `slot`: where the part
// goes, -1 where the block has the whole unit.  `note`: this thread writes down where the parts of a unit are.
template <typename F>
__device__ __forceinline__ void cache_walk(const CacheArgs& a, const CacheStart& s, bool note, F f) {
    CacheUnit u = s.u;
    int left = s.left, tile = s.tile;
    bool first = true;
#pragma unroll 1
    while (left > 0) {
        const int n = min(u.tiles - tile, left), slot = n == u.tiles ? -1 : 2 * (int)blockIdx.x + (first ? 0 : 1);
        if (note && tile == 0 && !a.whole)  // its first block says where its parts are
            a.units[(u.b * a.N + u.n) * a.row_tiles + u.rt] = make_int2(slot, 1 + (u.tiles - n + s.share - 1) / s.share);
        f(u, tile, n, slot);
        left -= n, tile = 0, first = false;
        if (left > 0) cache_next_unit(a, u);
    }
}

// ---- codes ----

__device__ __forceinline__ float cache_scale(uint32_t byte) { return __uint_as_float(byte << 23); }  // of bytes below 255
__device__ __forceinline__ float cache_row_scale(uint32_t byte) { return byte == 255u ? __uint_as_float(0x7fffffffu) : cache_scale(byte); }  // 255: NaN

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
