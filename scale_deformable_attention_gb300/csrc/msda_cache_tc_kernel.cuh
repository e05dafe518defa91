// msda_cache_tc_kernel.cuh -- attention over the paged cache of many rows a key head
// (drafted trees of shared heads, pieces of prompts) on the tensor cores
// (tcgen05, sm_103a), fp16 and bf16 queries, D a multiple of 16 up to 128.
//
//   S = Q K^T,  P = 2^(c S - m),  l += row sums,  O = 2^(m_old - m) O + P V
//
// A block an SM takes an equal share of the line of all tiles (see the plan in
// msda_cache.cuh), unit after unit: NQ tiles of up to 128 rows of one key head
// (tokens times the G heads that share it side by side) over tiles of 128 keys.
// Warps:
//   - one warpgroup a row tile on the scores, a thread a row: it reads S from
//     tensor memory and writes P (16 bits) back; O stays in tensor memory;
//   - one issues the TMA copies, a box of each page's rows that a tile holds, one
//     a row tile its products;
//   - unquantised: one clears the value rows that lie behind a sequence's last;
//   - 8 bits: a warpgroup turns the codes of a tile, a row a thread, into f16 rows
//     of the operands, the tile's largest scale being 2^7 (e4m3) or 2^5 (int8) of
//     theirs: the scores of the tile are multiplied by that scale of K, its P by
//     that of V over the largest met.  New tokens' rows go the same way.  Codes
//     2^22 or 2^29 below are still exact.  A key whose scale lies further below, as next
//     to one of nothing but a large channel, goes in at its own scale, and its
//     column of scores is multiplied by that (such scores were 0 from 2^25 on
//     otherwise); values of P V share a sum: codes are cut at 2^-31 (2^-29) of the
//     largest scale, scales below that are 0.
// bf16 queries of a quantised cache become f16 with a power of two a row.
//
// Measured, 16 heads on 4 of 128 channels over 8 x 65536 tokens: 64 rows a key head bf16 180 us (6.0 TB/s: memory), e4m3
// 180 us (a tile of 128 keys takes 2800 cycles: the scores' threads, one a scheduler, follow their own latencies); 256 rows
// bf16 255 us (1080 TFLOP/s, 3700 cycles a tile of two row tiles).  8 x 16384 tokens: 61, 69 and 90 us, of which 8 pass
// before the first product (code fetched, plan, queries) and 3 in the parts' writing.
//
// The reference m follows when a row's sum over a tile passes a limit, as in the
// dense forward: P is in f16 at most 49152 and m 2^8 below the maximum when it is
// looked for, in bf16 2^14.  f16 loses what lies 2^33 below the reference, and a
// row's output with it where one key outweighs the others while its value is
// small.  Such rows, one key with all but 1/128 of the sum so far, have a lower
// limit too: a tile below it gets an m of its own, O and l going up.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "msda_attention_tc.cuh"
#include "msda_cache.cuh"
#include "msda_cache_tc.cuh"
#include "msda_host.cuh"

namespace msda {

namespace {

template <bool OB>
struct CacheTcRange {
    static constexpr float kTop = OB ? 16384.f : 49152.f;  // the largest sum of a row over a tile; f16 holds 65504
    static constexpr float kBelow = OB ? 0.f : 8.f;        // m below the maximum: 128 equal ones add up to 2^15
    // f16, rows that one key outweighs (all but kAlone of the sum), as in the dense forward: the smallest sum of a tile, m below its
    // maximum when it goes down for one, and what keeps O under 2^127: l before, m's way
    static constexpr float kLow = 0x1p-7f, kBelowLow = 3.f, kMostL = 0x1p40f, kWay = 56.f, kAlone = 0x1p-7f;
};

template <int F, int NQ, int NC>
struct CacheTcCfg {  // stages are even in number: K has the even ones, V the odd ones
    static constexpr bool kCodes = F != kCacheSame;
    static_assert(!kCodes || NQ == 1, "codes: one row tile a block");
    static constexpr int kStages = NC == 1 ? (kCodes ? 6 : 8) : 4;  // ring of K and V operand tiles
    static constexpr int kRaw = !kCodes ? 0 : NC == 1 ? 6 : 4;                                  // ring of tiles of codes
    static constexpr int kThreads = NQ * 128 + 128 + (kCodes ? 256 : 0);
    static constexpr uint32_t kTileBytes = NC * kTcTile, kRawBytes = NC * 64 * 128;
    // Registers of a thread of the warpgroups on the scores, of the one that issues and of the two that convert: with codes the launch
    // of four warpgroups has 128 a thread, unquantised with two row tiles 168 of three; with one row tile 255, and no split.  (Codes at
    // 208/56/120, 224/48/120, 232/56/112, us: e4m3 piece of 1100 over 2 x 8191 of 64 channels 137.5, 130.5, 131.4; int8 tree of 16
    // over 16 x 16641 of 128 channels 101.6, 99.8, 101.9.)
    static constexpr int kUp = kCodes ? 224 : NQ == 1 ? 0 : 208, kDown = kCodes ? 48 : 88, kConvert = 120;
    static_assert(!kCodes || kUp + kDown + 2 * kConvert <= 512, "more registers than the launch has");
    static_assert(kCodes || NQ == 1 || NQ * kUp + kDown <= 504, "more registers than the launch has");
    // tensor memory: S (128 columns a row tile), P (64), O (64 or 128); two row tiles of up to 128 channels leave no room
    // for P: it lies over S, and the next S waits until P is used up
    static constexpr bool kOwnP = NC == 1 || NQ == 1;
    static constexpr uint32_t kP = kOwnP ? NQ * 128 : 0, kPStep = kOwnP ? 64 : 128;
    static constexpr uint32_t kO = kOwnP ? NQ * 192 : NQ * 128;
    static constexpr uint32_t kCols = NQ == 2 || NC == 2 ? 512 : 256;
    static constexpr size_t kSmem = (size_t)(NQ + kStages) * kTileBytes + (size_t)kRaw * kRawBytes + 1024;
    // The tile's largest scale in the operands' f16: 448 2^7 (new tokens: 65504) and 127 2^5 are within it, and so is the 1152 that
    // int8 codes pass by.  Binary places that a key may lie below and share it: codes stay exact (e4m3: 2^-9 2^(7 - 22), int8: 2^(5 - 29));
    // new tokens, whose rows then begin at 1, keep 2^-14 of their own largest in full.
    static constexpr int kLift = F == kCacheE4m3 ? 7 : 5;
    static constexpr int kApart = kLift + (F == kCacheE4m3 ? 15 : 24), kApartNew = kLift + 8;
};

struct CacheTcSync {
    uint64_t full[8], empty[8], raw_full[6], raw_empty[6];
    uint64_t cleared[8], q_full, q_empty, tops_full[2], s_full[2], s_free[2], p_full[2], pv_done[2], turn;
    uint32_t tmem, abort;
    uint32_t words[8][4];    // a tile's keys that are there
    float k_scale[8];        // 8 bits: scale of a tile's K, and the byte of that of its V
    uint32_t v_top[8];
    int k_far[8];            // tile i + 1: some of its keys have scales of their own
    alignas(16) uint32_t tops[2][2][4];  // of each warpgroup that converts, by turns: its warps' largest bytes
};

static_assert(CacheTcCfg<kCacheE4m3, 1, 2>::kSmem + sizeof(CacheTcSync) + sizeof(CacheStart) <= 227 * 1024, "more shared memory than a block has");

__device__ __forceinline__ void tc_tma_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// Of a new token's row: the byte of the power of two that brings its largest value to 2^8 or more; 255 where it holds an infinity or a NaN.
template <bool BF16, typename T>
__device__ __forceinline__ uint32_t cache_new_byte(const T* row, int D) {
    uint32_t top = 0;
#pragma unroll 4
    for (int d = 0; d < D; d += 8) {
        const uint4 y = *reinterpret_cast<const uint4*>(row + d);
        const uint32_t mm = 0x7fff7fffu;
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(y.x & mm, y.y & mm), __vmaxu2(y.z & mm, y.w & mm)));
    }
    top = max(top & 0xffffu, top >> 16);
    const float y = BF16 ? __uint_as_float(top << 16) : __half2float(__ushort_as_half((unsigned short)top));
    const int e = (int)(__float_as_uint(y) >> 23);
    return e == 255 ? 255u : (uint32_t)max(e - 8, 27);
}

// A unit's tiles of a block: cache tiles first, then those of the new tokens.
struct CacheSegment {
    CacheUnit u;
    int first, n, slot;  // tiles [first, first + n) of the unit
    int tail_keys;
};

// Calls f(segment) for each unit of the block; false ends it.  n is 0 for rows that see nothing.
template <typename F>
__device__ __forceinline__ void cache_segments(const CacheArgs& a, const CacheStart& start, bool note, F f) {
    bool ok = true;
    cache_walk(a, start, note, [&](const CacheUnit& u, int tile, int tiles, int slot) {
        if (!ok) return;
        CacheSegment s;
        s.u = u, s.first = tile, s.slot = slot;
        s.tail_keys = cache_tail_keys(a, u.rt, u.count);
        s.n = max(0, min(tiles, u.cache_tiles + (s.tail_keys + kTcRows - 1) / kTcRows - tile));
        ok = f(s);
    });
}

// Scores of a tile (at s_at in tensor memory) some of whose keys are at scales of their own: columns times these over 2^(most - 127).
// Worked out anew and outside of the loop, so that the way that most tiles take holds next to nothing of it (a table from the
// converting warps cost every tile 8 %; this 2 to 4: int8 92.9 -> 97.1 us for a tree of 16 over 16 x 16641 tokens).
template <bool BF16, int F>
__device__ __noinline__ void cache_tc_own_scales(const CacheArgs& a, const CacheSegment& sg, int tile, uint32_t most, uint32_t s_at) {
    using Cfg = CacheTcCfg<F, 1, 1>;
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    const int lane = threadIdx.x & 31;
    const CacheUnit& u = sg.u;
    const bool tail = tile >= u.cache_tiles;
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
        const int key = tile * kTcRows + c + lane, j = key - u.cache_tiles * kTcRows;
        uint32_t byte = 0;
        if (tail) {
            if (j < sg.tail_keys) byte = cache_new_byte<BF16>(static_cast<const T*>(a.nk) + u.b * a.nk_sb + j * a.nk_st + u.n * a.nk_sh, a.D);
        } else if (key < u.length) {
            const int page = cache_entry(a.c, u.b, key);
            if ((unsigned)page < (unsigned)a.c.pages) byte = a.c.ks[page * a.c.ks_sp + (key & (a.c.page - 1)) * a.c.ks_st + u.n * a.c.ks_sh];
        }
        const int below = (int)(most - byte);
        const float own = byte == 0u || below <= (tail ? Cfg::kApartNew : Cfg::kApart) ? 1.f : below > 126 ? 0.f : cache_scale(127 - below);
#pragma unroll 1
        for (int half = 0; half < 32; half += 16) {
            uint32_t x[16];
            tmem_ld16(x, s_at + c + half);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * __shfl_sync(0xffffffffu, own, half + k));
            tmem_st16(s_at + c + half, x);
        }
    }
    tmem_wait_st();
}

}  // namespace

template <bool BF16, int F, int NQ, int NC>
__global__ void __launch_bounds__(CacheTcCfg<F, NQ, NC>::kThreads, 1)
    msda_cache_tc_kernel(const __grid_constant__ CacheArgs a, const int box_rows, const __grid_constant__ CUtensorMap map_q,
                         const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                         const __grid_constant__ CUtensorMap map_nk, const __grid_constant__ CUtensorMap map_nv) {
    using Cfg = CacheTcCfg<F, NQ, NC>;
    constexpr bool CODES = Cfg::kCodes, OB = BF16 && !CODES, OWN_Q = BF16 && CODES;  // operands in bf16; queries turned into f16 by their rows' threads
    using Range = CacheTcRange<OB>;
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    constexpr int ST = Cfg::kStages;
    extern __shared__ unsigned char cache_tc_smem[];
    unsigned char* smem = cache_tc_smem + ((1024u - (tc_smem(cache_tc_smem) & 1023u)) & 1023u);
    unsigned char* q_tiles = smem;
    unsigned char* ring = smem + NQ * Cfg::kTileBytes;
    unsigned char* raw = ring + ST * Cfg::kTileBytes;
    __shared__ CacheTcSync sy;
    __shared__ CacheStart start;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int qpt = a.tile_rows / (NQ * a.G), rows = qpt * a.G;  // tokens and rows of a row tile

    if (warp == NQ * 4) {
        if (lane == 0) {
            for (int i = 0; i < 8; ++i) {
                tc_bar_init(tc_smem(&sy.full[i]), CODES ? 4 : 1);
                tc_bar_init(tc_smem(&sy.empty[i]), NQ + (!CODES && (i & 1) ? 1 : 0));  // values lie in the odd stages: the warp that clears lets them go too
                tc_bar_init(tc_smem(&sy.cleared[i]), 1);
            }
            for (int i = 0; i < 6; ++i) {
                tc_bar_init(tc_smem(&sy.raw_full[i]), 1);
                tc_bar_init(tc_smem(&sy.raw_empty[i]), 4);
            }
            tc_bar_init(tc_smem(&sy.q_full), OWN_Q ? NQ * 4 : 1);
            tc_bar_init(tc_smem(&sy.q_empty), NQ);
            tc_bar_init(tc_smem(&sy.turn), 1);
            for (int i = 0; i < 2; ++i) {
                tc_bar_init(tc_smem(&sy.tops_full[i]), 4);
                tc_bar_init(tc_smem(&sy.s_full[i]), 1);
                tc_bar_init(tc_smem(&sy.s_free[i]), 4);
                tc_bar_init(tc_smem(&sy.p_full[i]), 4);
                tc_bar_init(tc_smem(&sy.pv_done[i]), 1);
            }
            for (int i = 0; i < 8; ++i) sy.k_far[i] = 0;
            sy.abort = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            tc_prefetch_map(&map_q);
            tc_prefetch_map(&map_k);
            tc_prefetch_map(&map_v);
            if (!CODES && a.nk) {
                tc_prefetch_map(&map_nk);
                tc_prefetch_map(&map_nv);
            }
        }
    } else if (warp == NQ * 4 + 1) {
        tmem_alloc(tc_smem(&sy.tmem), Cfg::kCols);
    }
    if (warp == 0) {
        const CacheStart s = cache_start(a);
        if (lane == 0) start = s;
    }
    if (rows < kTcRows) {  // rows that no query fills hold zeros, not what was there
        const uint32_t words = (kTcRows - rows) * 8;
        for (uint32_t i = tid; i < NQ * NC * words; i += Cfg::kThreads) {
            const uint32_t c = i / words, w = i - c * words;
            *reinterpret_cast<uint4*>(q_tiles + c * kTcTile + rows * 128 + w * 16) = make_uint4(0, 0, 0, 0);
        }
        tc_fence_async();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sy.tmem;
    volatile uint32_t* abort = &sy.abort;
    unsigned* err = a.c.err;
    bool ok = true;

    if (warp < NQ * 4) {
        if constexpr (Cfg::kUp > 0) tc_regs_up<Cfg::kUp>();
        // ---- scores: row `row` of tile `t` ----
        const int t = warp >> 2, wl = warp & 3, row = wl * 32 + lane;
        const uint32_t lanes = (uint32_t)wl << 21;
        const uint32_t s_at = tmem + t * 128 + lanes, o_at = tmem + Cfg::kO + t * (NC * 64) + lanes;
        const uint32_t p_at = tmem + Cfg::kP + t * Cfg::kPStep + lanes;
        const int chunks = a.D / 16;
        const uint32_t first = lane == 0;
        int g0 = 0, p0 = 0;  // tiles before this segment, tiles of the cache so far
        cache_segments(a, start, tid == 0, [&](const CacheSegment& sg) {
            const CacheUnit& u = sg.u;
            const int tok = u.rt * NQ * qpt + t * qpt + row / a.G, h = u.n * a.G + row % a.G;
            const bool there = row < rows && tok < a.T, valid = there && tok < u.count;
            const bool warp_on = __any_sync(0xffffffffu, valid);
            float c2 = a.c2;
            if constexpr (OWN_Q) {
                if (sg.n > 0) {
                    // the row in f16, its largest brought to 2^14 or more (all of it in registers: its loads wait for one another no more)
                    const T* q = static_cast<const T*>(a.q) + u.b * a.q_sb + tok * a.q_st + h * a.q_sh;
                    uint4 x[NC * 8];
                    uint32_t top = 0;
#pragma unroll
                    for (int k = 0; k < NC * 8; ++k) x[k] = valid && k * 8 < a.D ? *reinterpret_cast<const uint4*>(q + k * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int k = 0; k < NC * 8; ++k) {
                        const uint32_t mm = 0x7fff7fffu;
                        top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[k].x & mm, x[k].y & mm), __vmaxu2(x[k].z & mm, x[k].w & mm)));
                    }
                    const int e = (int)(max(top & 0xffffu, top >> 16) >> 7);
                    const float up = e > 0 && e < 255 ? __uint_as_float((uint32_t)min(268 - e, 227) << 23) : 1.f;
                    c2 = a.c2 * (1.f / up);
                    if (row < rows) {
#pragma unroll
                        for (int k = 0; k < NC * 8; ++k) {
                            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                            uint32_t p[4];
#pragma unroll
                            for (int v = 0; v < 4; ++v) p[v] = tc_pack<false>(__uint_as_float(w[v] << 16) * up, __uint_as_float(w[v] & 0xffff0000u) * up);
                            *reinterpret_cast<uint4*>(q_tiles + (t * NC + k / 8) * kTcTile + row * 128 + (((k & 7) ^ (row & 7)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
                        }
                    }
                    tc_fence_async();
                    __syncwarp();
                    tc_bar_arrive_if(first, tc_smem(&sy.q_full));
                }
            }
            // reference, sum; f16: the sum of a tile that asks for a lower reference (0: none), the largest key's part of l
            float m = -attn_inf(), l = 0.f, low = 0.f, alone = 0.f;
            uint32_t v_ref = 0;
#pragma unroll 1
            for (int i = 0; i < sg.n; ++i) {
                const int gi = g0 + i, tile = sg.first + i;
                uint32_t w[4] = {~0u, ~0u, ~0u, ~0u};
                const bool tail = tile >= u.cache_tiles;
                if (tail) {
                    const int j0 = (tile - u.cache_tiles) * kTcRows, left = (valid ? u.count : 0) - j0;
#pragma unroll
                    for (int c = 0; c < 4; ++c) w[c] = tc_low_bits((a.mask ? left : min(left, tok + 1 - j0)) - 32 * c);
                    if (a.mask && valid) {
                        const uint8_t* mask = a.mask + u.b * a.mk_sb + tok * a.mk_sq + j0;
                        const int n = min(left, kTcRows);
                        const bool fours = (reinterpret_cast<uintptr_t>(mask) & 3) == 0;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t bits = 0;
                            if (fours) {
#pragma unroll 1
                                for (int k = 0; k < 32; k += 4) {
                                    const int j = c * 32 + k;
                                    uint32_t x = 0;
                                    if (j + 4 <= n) x = *reinterpret_cast<const uint32_t*>(mask + j);
                                    else
                                        for (int e = 0; e < 4; ++e)
                                            if (j + e < n) x |= (uint32_t)mask[j + e] << (8 * e);
#pragma unroll
                                    for (int e = 0; e < 4; ++e) bits |= ((x >> (8 * e)) & 255u ? 1u : 0u) << (k + e);
                                }
                            } else {
#pragma unroll 1
                                for (int k = 0; k < 32; ++k)
                                    if (c * 32 + k < n && mask[c * 32 + k]) bits |= 1u << k;
                            }
                            w[c] &= bits;
                        }
                    }
                }
                __syncwarp();
                if (!tc_bar_wait(tc_smem(&sy.s_full[t]), gi & 1, abort, err)) return false;
                tc_fence_after();
                if (warp_on) {
                    if constexpr (CODES) {
                        if (__builtin_expect(sy.k_far[gi & 7] == gi + 1, 0))
                            cache_tc_own_scales<BF16, F>(a, sg, tile, (__float_as_uint(sy.k_scale[gi & 7]) >> 23) + Cfg::kLift, s_at);
                    }
                    uint32_t s[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(s[c], s_at + c * 32);
                    tmem_wait_ld();
                    if constexpr (Cfg::kOwnP) {  // the next S may be written now
                        tc_fence_before();
                        tc_bar_arrive_if(first, tc_smem(&sy.s_free[t]));
                    }
                    if (!tail) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) w[c] = sy.words[p0 & 7][c];
                    }
                    if (__builtin_expect(__any_sync(0xffffffffu, (w[0] & w[1] & w[2] & w[3]) != 0xffffffffu), 0)) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!((w[c] >> k) & 1u)) s[c][k] = 0xff800000u;
                    }
                    float ct = c2, dv = 0.f;  // this tile's factor of the scores; binary places of its values' scale below v_ref
                    uint32_t v_old = v_ref;
                    if constexpr (CODES) {
                        ct = fmaxf(c2 * sy.k_scale[gi & 7], 1e-37f);  // never 0, which would make NaN of what is masked
                        const uint32_t vt = sy.v_top[gi & 7];
                        if (vt > v_ref) v_ref = vt;
                        dv = fmaxf((float)((int)vt - (int)v_ref), -60.f);  // beyond 2^-60 of the largest value nothing counts
                    }
                    const uint64_t cc = tc_two(ct, ct);
                    bool gone = false;
                    // P = 2^(c S - m) into tensor memory; the row's sum.  `wait`: the last P may still be read.
                    auto probabilities = [&](bool wait) {
                        const float ref = (m == -attn_inf() ? 0.f : m) - dv;
                        const uint64_t nref = tc_two(-ref, -ref);
                        uint64_t part[2] = {0, 0};
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t pk[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                float x0, x1;
                                tc_split(tc_fma2(tc_two(__uint_as_float(s[c][2 * k]), __uint_as_float(s[c][2 * k + 1])), cc, nref), x0, x1);
                                const float e0 = tc_ex2(x0), e1 = tc_ex2(x1);
                                part[k & 1] = tc_add2(part[k & 1], tc_two(e0, e1));
                                pk[k] = tc_pack<OB>(e0, e1);
                            }
                            if (c == 0 && wait) {
                                gone = !tc_bar_wait(tc_smem(&sy.pv_done[t]), (gi - 1) & 1, abort, err);
                                tc_fence_after();
                            }
                            tmem_st16(p_at + c * 16, pk);
                        }
                        float s0, s1;
                        tc_split(tc_add2(part[0], part[1]), s0, s1);
                        return s0 + s1;
                    };
                    // One place for the exponentials (code that is fetched first takes longer than it runs): against the reference at
                    // hand, and once more where that is none yet or a sum asks for another.
                    bool renew = (CODES && v_ref != v_old && i > 0) || __any_sync(0xffffffffu, valid && m == -attn_inf());
                    bool fresh = Cfg::kOwnP && i > 0;  // the last P is not known to be used up
                    float sum = 0.f;
#pragma unroll 1
                    for (int pass = 0; pass < 2; ++pass) {
                        if (__builtin_expect(renew, 0)) {
                            if (fresh) {
                                gone = !tc_bar_wait(tc_smem(&sy.pv_done[t]), (gi - 1) & 1, abort, err);
                                tc_fence_after();
                                fresh = false;
                            }
                            float mx[4];
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                mx[c] = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
                                for (int k = 2; k < 32; k += 2)
                                    mx[c] = tc_max3(mx[c], __uint_as_float(s[c][k]), __uint_as_float(s[c][k + 1]));
                            }
                            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * ct;
                            float next = fmaxf(m, top - Range::kBelow);
                            if constexpr (!OB) {
                                if (next > m) alone = exp2f(Range::kBelow);
                                if (low > 0.f && top < m - 6.f && top > m - Range::kWay) next = top - Range::kBelowLow;
                            }
                            const float f = next == m ? 1.f : tc_ex2(m - next);
                            if (!OB && next < m) alone *= f;
                            m = next;
                            l *= f;
                            if (i > 0) {
                                float fo = f;
                                if constexpr (CODES) fo *= v_ref - v_old > 126 ? 0.f : cache_scale(127 + v_old - v_ref);
#pragma unroll 1
                                for (int c = 0; c < chunks; ++c) {
                                    uint32_t o[16];
                                    tmem_ld16(o, o_at + c * 16);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fo);
                                    tmem_st16(o_at + c * 16, o);
                                }
                            }
                            if constexpr (CODES) v_old = v_ref;
                            pass = 1;  // the reference is the tile's own: no sum can ask for another
                        }
                        sum = probabilities(fresh);
                        fresh = false;
                        const bool fits = sum <= Range::kTop;
                        if constexpr (CODES) sum *= exp2f(-dv);
                        if constexpr (!OB) {
                            if (renew) low = l + sum - alone < alone * Range::kAlone && l < Range::kMostL ? Range::kLow : 0.f;
                        }
                        renew = __any_sync(0xffffffffu, valid && !(fits && (OB || sum >= low)));
                        if (!renew) break;
                    }
                    if (__builtin_expect(gone, 0)) return false;
                    l += sum;
                    tmem_wait_st();
                    tc_fence_before();
                } else if constexpr (Cfg::kOwnP) {
                    tc_bar_arrive_if(first, tc_smem(&sy.s_free[t]));
                    // a warp without rows may not run a tile ahead of the others: its arrival would count for theirs
                    if (i > 0 && !tc_bar_wait(tc_smem(&sy.pv_done[t]), (gi - 1) & 1, abort, err)) return false;
                }
                p0 += tail ? 0 : 1;
                __syncwarp();
                tc_bar_arrive_if(first, tc_smem(&sy.p_full[t]));
            }
            // ---- output ----
            if (sg.n > 0) {
                if (!tc_bar_wait(tc_smem(&sy.pv_done[t]), (g0 + sg.n - 1) & 1, abort, err)) return false;
                tc_fence_after();
            }
            g0 += sg.n;
            if (!__any_sync(0xffffffffu, there)) return true;
            const bool none = l == 0.f || !valid;
            const float inv = none ? 0.f : 1.f / l, unit = !CODES ? 1.f : v_ref > Cfg::kLift ? cache_scale(v_ref - Cfg::kLift) : 0.f;  // one after the other: their product may be below binary32
            const float l2 = none ? -attn_inf() : m + log2f(l);
            const long long at = (long long)sg.slot * a.tile_rows + t * rows + row;
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                uint32_t o[16];
                if (sg.n > 0 && warp_on) {
                    tmem_ld16(o, o_at + c * 16);
                    tmem_wait_ld();
                }
                if (!there) continue;
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = none ? 0u : __float_as_uint(__uint_as_float(o[k]) * inv * unit);
                if (sg.slot >= 0) {
                    float* out = a.part_o + at * a.D + c * 16;
#pragma unroll
                    for (int k = 0; k < 4; ++k) reinterpret_cast<uint4*>(out)[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                } else {
                    T* out = static_cast<T*>(a.out) + (((long long)u.b * a.T + tok) * a.M + h) * a.D + c * 16;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = tc_pack<BF16>(__uint_as_float(o[8 * k + 2 * e]), __uint_as_float(o[8 * k + 2 * e + 1]));
                        reinterpret_cast<uint4*>(out)[k] = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
            if (there) {
                if (sg.slot >= 0) a.part_l2[at] = l2;
                else a.lse[((long long)u.b * a.M + h) * a.T + tok] = l2 * kLn2;
            }
            tc_fence_before();
            return true;
        });
        ok = !*abort;
    } else if (warp < NQ * 4 + 4) {
        if constexpr (Cfg::kUp > 0) tc_regs_down<Cfg::kDown>();
        const int role = warp - NQ * 4;
        if (role == 0) {
            // ---- copies (all lanes: a box of rows each) ----
            const int boxes = kTcRows / box_rows;
            const uint32_t qbar = tc_smem(&sy.q_full);
            int g0 = 0, p0 = 0, qs = 0;  // tiles, tiles of the cache, queries so far
            cache_segments(a, start, false, [&](const CacheSegment& sg) {
                const CacheUnit& u = sg.u;
                if (sg.n == 0) return true;
                if constexpr (!OWN_Q) {
                    if (qs > 0 && !tc_bar_wait(tc_smem(&sy.q_empty), (qs - 1) & 1, abort, err)) return false;
                    if (lane == 0) {
                        tc_bar_expect(qbar, NQ * NC * rows * 128);
                        for (int t = 0; t < NQ; ++t)
                            for (int c = 0; c < NC; ++c)
                                tc_tma_5d(tc_smem(q_tiles) + (t * NC + c) * kTcTile, &map_q, qbar, c * 64, 0, (u.rt * NQ + t) * qpt, u.n, u.b);
                    }
                    ++qs;
                }
                auto entry_of = [&](int i) {  // of this lane's box at tile sg.first + i
                    const int tile = sg.first + i, token = tile * kTcRows + lane * box_rows;
                    return i < sg.n && lane < boxes && tile < u.cache_tiles && token < u.length ? cache_entry(a.c, u.b, token) : kCacheNoPage;
                };
                int entry = entry_of(0), entry1 = entry_of(1);
                for (int i = 0; i < sg.n; ++i) {
                    const int gi = g0 + i, tile = sg.first + i, mine = cache_page_of(a.c, entry);
                    entry = entry1, entry1 = entry_of(i + 2);
                    const bool tail = tile >= u.cache_tiles;
                    if (!tail) {
                        // eight places by turns, counted in tiles of the cache: those ahead are in the rings (tiles of new tokens pass
                        // this warp by where the cache holds codes, any number of them)
                        const uint32_t good = __ballot_sync(0xffffffffu, mine >= 0);
                        const int x = lane & 3;  // keys 32 x to 32 x + 31
                        const uint32_t pages = box_rows >= 32 ? ((good >> (x * 32 / box_rows)) & 1u ? ~0u : 0u)
                                                              : ((good >> (2 * x)) & 1u ? 0xffffu : 0u) | ((good >> (2 * x + 1)) & 1u ? 0xffff0000u : 0u);
                        if (lane < 4) sy.words[p0 & 7][x] = pages & tc_low_bits(u.length - tile * kTcRows - 32 * x);
                        __syncwarp();
                    }
                    const int ring_n = CODES ? Cfg::kRaw : ST;
                    if (tail && CODES) continue;  // the converters read them
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const int idx = 2 * (CODES ? p0 : gi) + kv, st = idx % ring_n;
                        uint64_t* full = CODES ? sy.raw_full : sy.full;
                        uint64_t* empty = CODES ? sy.raw_empty : sy.empty;
                        if (idx >= ring_n && !tc_bar_wait(tc_smem(&empty[st]), (idx / ring_n - 1) & 1, abort, err)) return false;
                        const uint32_t bar = tc_smem(&full[st]);
                        const uint32_t dst = CODES ? tc_smem(raw) + st * Cfg::kRawBytes : tc_smem(ring) + st * Cfg::kTileBytes;
                        if (lane == 0) tc_bar_expect(bar, CODES ? Cfg::kRawBytes : Cfg::kTileBytes);
                        __syncwarp();
                        if (tail) {
                            if (lane < NC) tc_tma_4d(dst + lane * kTcTile, kv ? &map_nv : &map_nk, bar, lane * 64, u.n, (tile - u.cache_tiles) * kTcRows, u.b);
                        } else if (lane < boxes) {
                            const int pg = mine < 0 ? a.c.pages : mine, at = mine < 0 ? 0 : (tile * kTcRows + lane * box_rows) & (a.c.page - 1);
                            if constexpr (CODES) {
                                tc_tma_4d(dst + lane * box_rows * (NC * 64), kv ? &map_v : &map_k, bar, 0, u.n, at, pg);
                            } else {
                                for (int c = 0; c < NC; ++c)
                                    tc_tma_4d(dst + c * kTcTile + lane * box_rows * 128, kv ? &map_v : &map_k, bar, c * 64, u.n, at, pg);
                            }
                        }
                    }
                    p0 += tail ? 0 : 1;
                }
                g0 += sg.n;
                return true;
            });
        } else if (role == 1 || (NQ == 2 && role == 3)) {
            // ---- products of row tile t ----
            const int t = role >> 1;
            const uint32_t on = tc_elect();
            const uint32_t id_qk = tc_idesc(OB, false, false, 128, 128);
            const int steps = a.D / 16;
            const uint32_t id_pv = tc_idesc(OB, false, true, 128, steps * 16);
            const uint32_t ring_at = tc_smem(ring);
            const uint64_t q_desc = tc_desc(tc_smem(q_tiles) + t * Cfg::kTileBytes, 16, 1024);
            const uint32_t s_at = tmem + t * 128, o_at = tmem + Cfg::kO + t * (NC * 64);
            const uint32_t p_at = tmem + Cfg::kP + t * Cfg::kPStep;
            auto product_s = [&](int st) {
                const uint64_t k_desc = tc_desc(ring_at + st * Cfg::kTileBytes, 16, 1024);
#pragma unroll
                for (int k = 0; k < NC * 4; ++k) {  // 16 channels: 32 bytes further, 64: the next tile
                    const uint64_t off = ((k >> 2) * kTcTile + (k & 3) * 32) >> 4;
                    if (k < steps) tc_mma_ss(on, s_at, q_desc + off, k_desc + off, id_qk, k > 0);
                }
                tc_commit(on, tc_smem(&sy.s_full[t]));
                tc_commit(on, tc_smem(&sy.empty[st]));
            };
            int g0 = 0, qs = 0;
            uint32_t clears = 0;  // a bit a stage: which phase of its `cleared` is next
            cache_segments(a, start, false, [&](const CacheSegment& sg) {
                const CacheUnit& u = sg.u;
                if (sg.n == 0) return true;
                if (!tc_bar_wait(tc_smem(&sy.q_full), qs & 1, abort, err)) return false;
                ++qs;
                // K of tile gi, when S may be written
                auto next_s = [&](int gi) {
                    const int idx = 2 * gi, st = idx % ST;
                    if (!tc_bar_wait(tc_smem(&sy.full[st]), (idx / ST) & 1, abort, err)) return false;
                    // the scale of the tile's values, which the scores' threads read, comes from another warpgroup than that of its keys
                    if (CODES && !tc_bar_wait(tc_smem(&sy.full[(idx + 1) % ST]), ((idx + 1) / ST) & 1, abort, err)) return false;
                    if (Cfg::kOwnP && gi > 0 && !tc_bar_wait(tc_smem(&sy.s_free[t]), (gi - 1) & 1, abort, err)) return false;
                    tc_fence_after();
                    product_s(st);
                    return true;
                };
                // P over S: the second row tile starts when the first has worked out its first P
                if (!Cfg::kOwnP && t == 1 && g0 == 0 && !tc_bar_wait(tc_smem(&sy.turn), 0, abort, err)) return false;
                if (!next_s(g0)) return false;
                for (int i = 0; i < sg.n; ++i) {
                    const int gi = g0 + i, iv = 2 * gi + 1, sv = iv % ST, tile = sg.first + i;
                    const bool more = i + 1 < sg.n;
                    if (Cfg::kOwnP && more && !next_s(gi + 1)) return false;
                    if (!tc_bar_wait(tc_smem(&sy.full[sv]), (iv / ST) & 1, abort, err)) return false;
                    if constexpr (!CODES) {
                        const int left = tile < u.cache_tiles ? u.length - tile * kTcRows : u.count - (tile - u.cache_tiles) * kTcRows;
                        if (left < kTcRows) {
                            if (!tc_bar_wait(tc_smem(&sy.cleared[sv]), (clears >> sv) & 1, abort, err)) return false;
                            clears ^= 1u << sv;
                        }
                    }
                    if (!tc_bar_wait(tc_smem(&sy.p_full[t]), gi & 1, abort, err)) return false;
                    tc_fence_after();
                    if (!Cfg::kOwnP && NQ == 2 && t == 0 && gi == 0) tc_bar_arrive_if(on, tc_smem(&sy.turn));
                    const uint64_t v_desc = tc_desc(ring_at + sv * Cfg::kTileBytes, kTcTile, 1024);
#pragma unroll
                    for (int k = 0; k < 8; ++k)  // 16 keys: two atoms further
                        tc_mma_ts(on, o_at, p_at + k * 8, v_desc + ((k * 2048) >> 4), id_pv, i > 0 || k > 0);
                    tc_commit(on, tc_smem(&sy.pv_done[t]));
                    tc_commit(on, tc_smem(&sy.empty[sv]));
                    if (!Cfg::kOwnP && more && !next_s(gi + 1)) return false;
                }
                if constexpr (!OWN_Q) tc_commit(on, tc_smem(&sy.q_empty));
                g0 += sg.n;
                return true;
            });
        } else if (role == 2 && !CODES) {
            // ---- value rows behind the last ----
            int g0 = 0;
            cache_segments(a, start, false, [&](const CacheSegment& sg) {
                const CacheUnit& u = sg.u;
                for (int i = 0; i < sg.n; ++i) {
                    // every tile is waited for, in its turn: a barrier tells only the last phase from the one under way
                    const int tile = sg.first + i, idx = 2 * (g0 + i) + 1, st = idx % ST;
                    const int left = tile < u.cache_tiles ? u.length - tile * kTcRows : u.count - (tile - u.cache_tiles) * kTcRows;
                    if (!tc_bar_wait(tc_smem(&sy.full[st]), (idx / ST) & 1, abort, err)) return false;
                    if (left < kTcRows) {
                        const uint32_t w[4] = {tc_low_bits(left), tc_low_bits(left - 32), tc_low_bits(left - 64), tc_low_bits(left - 96)};
                        tc_clear_rows<NC>(ring + st * Cfg::kTileBytes, w, lane);
                        tc_fence_async();
                        __syncwarp();
                        if (lane == 0) tc_bar_arrive(tc_smem(&sy.cleared[st]));
                    }
                    __syncwarp();
                    if (lane == 0) tc_bar_arrive(tc_smem(&sy.empty[st]));
                }
                g0 += sg.n;
                return true;
            });
        }
        __syncwarp();
        ok = !*abort;
    } else if constexpr (CODES) {
        tc_regs_down<Cfg::kConvert>();
        // ---- codes to f16 operands: row `row` of each tile, one warpgroup for K and one for V (one for both took 2.2 us a tile of 128
        // channels, these 1.4) ----
        const int kv = (warp - NQ * 4 - 4) >> 2, cw = (warp - NQ * 4 - 4) & 3, row = cw * 32 + lane;
        int g0 = 0, r0 = 0;
        cache_segments(a, start, false, [&](const CacheSegment& sg) {
            const CacheUnit& u = sg.u;
            const uint8_t* scales = kv ? a.c.vs + u.n * a.c.vs_sh : a.c.ks + u.n * a.c.ks_sh;
            const long long s_page = kv ? a.c.vs_sp : a.c.ks_sp, s_token = kv ? a.c.vs_st : a.c.ks_st;
            const T* fresh = kv ? static_cast<const T*>(a.nv) + u.b * a.nv_sb + u.n * a.nv_sh : static_cast<const T*>(a.nk) + u.b * a.nk_sb + u.n * a.nk_sh;
            const long long f_token = kv ? a.nv_st : a.nk_st;
            const int apart = kv ? 300 : Cfg::kApart;  // values share a sum: no scales of their own
            auto entry_of = [&](int i) {  // of this row at tile sg.first + i
                const int token = (sg.first + i) * kTcRows + row;
                return i < sg.n && sg.first + i < u.cache_tiles && token < u.length ? cache_entry(a.c, u.b, token) : kCacheNoPage;
            };
            // its byte, untouched until its tile comes (any arithmetic would wait for it here)
            uint32_t ahead = 0;
            bool here = false;
            auto read_byte = [&](int i, int entry) {
                here = (unsigned)entry < (unsigned)a.c.pages;  // the warp that copies tells of bad ones
                const int page = here ? entry : 0, place = ((sg.first + i) * kTcRows + row) & (a.c.page - 1);
                ahead = 0;
                if (here) ahead = scales[page * s_page + place * s_token];
            };
            int entry = entry_of(0), entry1 = entry_of(1), entry2 = entry_of(2);
            read_byte(0, entry);
#pragma unroll 1
            for (int i = 0; i < sg.n; ++i) {
                const int gi = g0 + i, tile = sg.first + i;
                const bool tail = tile >= u.cache_tiles;
                const int j = (tile - u.cache_tiles) * kTcRows + row;  // new token (tail)
                bool there = here;
                uint32_t byte = ahead;  // of a new token's row: the byte that brings its largest value to 2^8 or more
                read_byte(i + 1, entry1);
                entry1 = entry2, entry2 = entry_of(i + 3);
                if (tail) {
                    there = j < sg.tail_keys;
                    byte = there ? cache_new_byte<BF16>(fresh + j * f_token, a.D) : 27u;
                }
                // the tile's largest scale, and where it is read
                const uint32_t mine = __reduce_max_sync(0xffffffffu, there && byte != 255u ? byte : 0u);
                if (lane == 0) {
                    sy.tops[kv][gi & 1][cw] = mine;
                    tc_bar_arrive(tc_smem(&sy.tops_full[kv]));
                }
                if (!tc_bar_wait(tc_smem(&sy.tops_full[kv]), gi & 1, abort, err)) return false;
                const uint4 all = *reinterpret_cast<const uint4*>(sy.tops[kv][gi & 1]);
                const uint32_t most = max(max(all.x, all.y), max(all.z, all.w));
                if (row == 0) {
                    if (kv) sy.v_top[gi & 7] = most;
                    else sy.k_scale[gi & 7] = most > Cfg::kLift ? cache_scale(most - Cfg::kLift) : 0.f;
                }
                const int idx = 2 * gi + kv, st = idx % ST;
                unsigned char* to = ring + st * Cfg::kTileBytes + row * 128;
                if (!tail) {
                    const int ri = 2 * r0 + kv, rs = ri % Cfg::kRaw;
                    if (!tc_bar_wait(tc_smem(&sy.raw_full[rs]), (ri / Cfg::kRaw) & 1, abort, err)) return false;
                    if (idx >= ST && !tc_bar_wait(tc_smem(&sy.empty[st]), (idx / ST - 1) & 1, abort, err)) return false;
                    const unsigned char* from = raw + rs * Cfg::kRawBytes + row * (NC * 64);
                    // 2^(byte - most + lift) in f16; a row that held no numbers: NaN; byte 0: zeros
                    const int below = (int)(most - byte);
                    const bool far = below > apart && byte != 0u;  // goes in at its own scale
                    const float f = byte == 255u ? __uint_as_float(0x7fffffffu) : far ? cache_scale(127 + Cfg::kLift) : byte == 0u || below > 126 ? 0.f : cache_scale(127 + Cfg::kLift - below);
                    const __half2 scale = __half2half2(__float2half_rn(f));
                    const __half2 off = __hmul2(scale, __half2half2(__ushort_as_half(0xe480)));  // -1152
#pragma unroll 1
                    for (int c0 = 0; c0 < NC * 4; c0 += 4) {  // 64 codes at a time, their loads first
                        uint4 y[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            y[c] = *reinterpret_cast<const uint4*>(from + ((NC == 2 ? (c0 + c) ^ (row & 7) : c ^ ((row >> 1) & 3)) << 4));
                        unsigned char* at = to + (c0 / 4) * kTcTile;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t w[4] = {y[c].x, y[c].y, y[c].z, y[c].w};
                            uint32_t p[8];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                __half2 y0, y1;
                                if constexpr (F == kCacheE4m3) {
                                    uint32_t lo, hi;
                                    cache_four_f16<F>(w[k], lo, hi);
                                    y0 = __hmul2(*reinterpret_cast<const __half2*>(&lo), scale), y1 = __hmul2(*reinterpret_cast<const __half2*>(&hi), scale);
                                } else {  // (1024 + u) s - 1152 s, exact
                                    const uint32_t v = w[k] ^ 0x80808080u, lo = __byte_perm(v, 0x64646464u, 0x4140), hi = __byte_perm(v, 0x64646464u, 0x4342);
                                    y0 = __hfma2(*reinterpret_cast<const __half2*>(&lo), scale, off), y1 = __hfma2(*reinterpret_cast<const __half2*>(&hi), scale, off);
                                }
                                p[2 * k] = there ? *reinterpret_cast<const uint32_t*>(&y0) : 0u;  // behind the last row: zeros, whatever lies there
                                p[2 * k + 1] = there ? *reinterpret_cast<const uint32_t*>(&y1) : 0u;
                            }
                            *reinterpret_cast<uint4*>(at + (((2 * c) ^ (row & 7)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
                            *reinterpret_cast<uint4*>(at + (((2 * c + 1) ^ (row & 7)) << 4)) = make_uint4(p[4], p[5], p[6], p[7]);
                        }
                    }
                    tc_fence_async();
                    __syncwarp();
                    if (far) sy.k_far[gi & 7] = gi + 1;
                    __syncwarp();
                    if (lane == 0) {
                        tc_bar_arrive(tc_smem(&sy.full[st]));
                        tc_bar_arrive(tc_smem(&sy.raw_empty[rs]));
                    }
                } else {
                    if (idx >= ST && !tc_bar_wait(tc_smem(&sy.empty[st]), (idx / ST - 1) & 1, abort, err)) return false;
                    const T* p = fresh + j * f_token;
                    const bool far = kv == 0 && there && byte + Cfg::kApartNew < most;
                    const float f = most == 0u ? 0.f : cache_scale(254u + Cfg::kLift - (far ? byte : most));
#pragma unroll 2
                    for (int d = 0; d < NC * 64; d += 8) {
                        uint4 y = make_uint4(0, 0, 0, 0);
                        if (there && d < a.D) {
                            const uint4 v4 = *reinterpret_cast<const uint4*>(p + d);
                            const uint32_t w[4] = {v4.x, v4.y, v4.z, v4.w};
                            uint32_t z[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float2 v;
                                if constexpr (BF16) v = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
                                else v = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
                                z[k] = tc_pack<false>(v.x * f, v.y * f);
                            }
                            y = make_uint4(z[0], z[1], z[2], z[3]);
                        }
                        *reinterpret_cast<uint4*>(to + (d / 64) * kTcTile + ((((d / 8) & 7) ^ (row & 7)) << 4)) = y;
                    }
                    tc_fence_async();
                    if (far) sy.k_far[gi & 7] = gi + 1;
                    __syncwarp();
                    if (lane == 0) tc_bar_arrive(tc_smem(&sy.full[st]));
                }
                if (!tail) ++r0;
            }
            g0 += sg.n;
            return true;
        });
        __syncwarp();
        ok = !*abort;
    }
    if (!ok) tc_drain();
    tc_fence_before();
    __syncthreads();
    if (warp == NQ * 4 + 1) tmem_dealloc(tmem, Cfg::kCols);
}

// ---- host ----

namespace {

using EncodeTiled = PFN_cuTensorMapEncodeTiled_v12000;

// Four dimensions (channel, head, row, outer) of `es` bytes an element; boxes of 64 channels (codes: all) x 1 x box_rows x 1.
bool map4(const void* base, int es, bool bf16, int64_t D, int inner, int64_t heads, int64_t rows, int64_t outer, int64_t sh, int64_t sr, int64_t so,
          int box_rows, CUtensorMap* map) {
    EncodeTiled f = reinterpret_cast<EncodeTiled>(tensor_map_encoder());
    if (!f) return false;
    auto bytes = [es](int64_t n, int64_t stride) { return (cuuint64_t)(n > 1 ? stride * es : 16); };
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows, (cuuint64_t)outer};
    const cuuint64_t strides[3] = {bytes(heads, sh), bytes(rows, sr), bytes(outer, so)};
    const cuuint32_t box[4] = {(cuuint32_t)inner, 1u, (cuuint32_t)box_rows, 1u};
    const cuuint32_t one[4] = {1u, 1u, 1u, 1u};
    return f(map, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
             const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             inner * es == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Queries [B, T, heads, D] as (channel, head of the group, token, key head, sequence); boxes of 64 channels x G heads x `tokens`.
bool map_queries(const CacheArgs& a, bool bf16, int tokens, CUtensorMap* map) {
    EncodeTiled f = reinterpret_cast<EncodeTiled>(tensor_map_encoder());
    if (!f) return false;
    auto bytes = [](int64_t n, int64_t stride) { return (cuuint64_t)(n > 1 ? stride * 2 : 16); };
    const cuuint64_t dims[5] = {(cuuint64_t)a.D, (cuuint64_t)a.G, (cuuint64_t)a.T, (cuuint64_t)a.N, (cuuint64_t)a.B};
    const cuuint64_t strides[4] = {bytes(a.G, a.q_sh), bytes(a.T, a.q_st), bytes(a.N, a.G * a.q_sh), bytes(a.B, a.q_sb)};
    const cuuint32_t box[5] = {64u, (cuuint32_t)a.G, (cuuint32_t)tokens, 1u, 1u};
    const cuuint32_t one[5] = {1u, 1u, 1u, 1u, 1u};
    return f(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, const_cast<void*>(a.q), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BF16, int F, int NQ, int NC>
cudaError_t tc_go(const CacheArgs& a, int grid, cudaStream_t st) {
    using Cfg = CacheTcCfg<F, NQ, NC>;
    const int qpt = a.tile_rows / (NQ * a.G), box_rows = a.c.page < kTcRows ? a.c.page : kTcRows;
    const int es = F == kCacheSame ? 2 : 1, inner = F == kCacheSame ? 64 : NC * 64;
    CUtensorMap mq, mk, mv, mnk, mnv;
    const bool fresh = F == kCacheSame && a.nk;
    const bool cache = a.c.longest > 0;  // else every length is 0: there are no tiles of the cache, and its maps are not used
    if (!map_queries(a, BF16, qpt, &mq) ||
        (cache && (!map4(a.c.k, es, BF16, a.D, inner, a.N, a.c.page, a.c.pages, a.c.k_sh, a.c.k_st, a.c.k_sp, box_rows, &mk) ||
                   !map4(a.c.v, es, BF16, a.D, inner, a.N, a.c.page, a.c.pages, a.c.v_sh, a.c.v_st, a.c.v_sp, box_rows, &mv))) ||
        (fresh && (!map4(a.nk, 2, BF16, a.D, 64, a.N, a.T, a.B, a.nk_sh, a.nk_st, a.nk_sb, kTcRows, &mnk) ||
                   !map4(a.nv, 2, BF16, a.D, 64, a.N, a.T, a.B, a.nv_sh, a.nv_st, a.nv_sb, kTcRows, &mnv))))
        return cudaErrorInvalidValue;
    if (!cache) mk = mv = mq;
    if (!fresh) mnk = mnv = mq;
    static SmemSeen seen;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(&msda_cache_tc_kernel<BF16, F, NQ, NC>), Cfg::kSmem, seen);
    if (e != cudaSuccess) return e;
    msda_cache_tc_kernel<BF16, F, NQ, NC><<<grid, Cfg::kThreads, Cfg::kSmem, st>>>(a, box_rows, mq, mk, mv, mnk, mnv);
    return cudaGetLastError();
}
}  // namespace

template <bool BF16, int F>
cudaError_t launch_cache_tc(const CacheArgs& a, int nq, int grid, cudaStream_t st) {
    if constexpr (F == kCacheSame) {
        if (nq == 2) return a.D > 64 ? tc_go<BF16, F, 2, 2>(a, grid, st) : tc_go<BF16, F, 2, 1>(a, grid, st);
    }
    return a.D > 64 ? tc_go<BF16, F, 1, 2>(a, grid, st) : tc_go<BF16, F, 1, 1>(a, grid, st);
}

}  // namespace msda
