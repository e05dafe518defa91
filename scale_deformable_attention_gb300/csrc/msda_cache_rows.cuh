// msda_cache_rows.cuh -- attention over the paged cache of few rows a key head
// (queries times the heads that share the key head: tiles of 16 or 32).
//
//   s = c Q K^T,  P = 2^(s - m),  l += row sums,  O += P V
//
// What bounds it: reading K and V once.  A block of four warps takes a share of
// the keys of one key head (see the plan); a warp walks its own steps of KS keys
// with its own reference m and sum l, fed by its own ring in shared memory
// (cp.async, no barrier of the block inside the loop), and the warps are joined
// at the end in a fixed order.  The products are mma.sync m16n8k16: with 16 rows
// tcgen05 would fill an eighth of its tile of 128, and its chain of product,
// tensor memory, exponentials and product takes 1 us a tile.
//
// Which channel a place of a product's contraction holds is free as long as both
// operands agree.  So a lane reads 16 bytes of a key in one load and uses them
// for 4, 2 or 1 steps of K, and of V it reads the same 16 bytes of channels of
// the four keys that it has in a step of 16, which one byte permutation a
// register brings next to each other: no transposing load.  16-byte chunks of a
// row are swizzled by the row so that both reads are free of bank conflicts.
//
// Measured, one new token of 16 heads on 4 of 128 channels: 8 x 65536 tokens bf16 169 us (6.3 TB/s), e4m3 119 us (4.6 TB/s:
// half the bytes, the same products and exponentials); 8 x 16384: 53 and 44 us, binary32 114 and, over e4m3, 69.  About 8 us of each pass before a
// block's first product: code that runs once costs some 9 cycles an instruction to fetch (plan 2.5 us, first
// copies 2.5, queries 1.2), so copies, products and exponentials stand in one place of the code each.
//
// Types.  16 bits: as they are.  8 bits: codes are whole f16 values, so the
// product is of f16 whatever the queries are; these are scaled by a power of two
// a row (bf16 has fewer bits than f16, binary32 takes two pieces), the scales of
// keys multiply the scores, those of values the probabilities, relative to the
// largest that the warp has met.  binary32: three bf16 pieces a value, six
// products, the small ones first.  A tensor core cuts its sums off: in binary32
// the outputs of 16 keys are summed anew and added in binary32 (480 sequences of
// 67200 tokens, e4m3, positive values: low by 5e-5 without that); scores run
// through the D / 16 products of a key in one sum.  P is rounded to 16 bits for its product (binary32: 2 pieces of f16
// or 3 of bf16).  f16 P: m lies 2^12 below the row's maximum when it was looked
// for, and is looked for again when a lane's P of a row add up to more than 1.5 2^15:
// a P is off by half a step or 2^-37 of the row's largest.  That loses a row's
// output where one key outweighs the others while its value is small; rows of
// which one key has all but 1/128 take a lower m for steps that fall far below.
#pragma once

#include "msda_cache.cuh"
#include "msda_host.cuh"

namespace msda {

constexpr int kCacheWarps = 4;

template <typename T>
struct CacheType;
template <>
struct CacheType<float> {
    static constexpr int code = 0;
    static __device__ __forceinline__ float put(float x) { return x; }
};
template <>
struct CacheType<__half> {
    static constexpr int code = 1;
    static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};
template <>
struct CacheType<__nv_bfloat16> {
    static constexpr int code = 2;
    static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};

// How a product runs for queries T over rows of format F: in bf16 or f16, and in how many pieces.
template <typename T, int F>
struct CacheProduct {
    static constexpr bool f32 = sizeof(T) == 4;
    static constexpr bool bf16 = F == kCacheSame && CacheType<T>::code != 1;
    static constexpr int es = F == kCacheSame ? (int)sizeof(T) : 1;
    static constexpr int qp = !f32 ? 1 : F == kCacheSame ? 3 : 2, kp = f32 && F == kCacheSame ? 3 : 1, pp = qp;
    // m below the maximum, in binary places, and what a lane's probabilities of a row may add up to in a step before m follows: f16 holds
    // 65504, eight equal ones at the maximum are 2^15
    static constexpr float below = bf16 ? 0.f : 12.f, most = bf16 ? 16384.f : 49152.f;
    // f16, rows that one key outweighs (all but `alone` of the sum): the smallest sum of a lane's keys, how far a step's maximum lies
    // below m before m goes down for it, m below it then (binary32 over codes: two pieces, that is 2^-24 of a sum of 4 or more), and what
    // keeps O under 2^127: l before, m's way
    static constexpr float low = f32 ? 4.f : 0x1p-7f, drop = f32 ? 0.f : 6.f, below_low = f32 ? 8.f : 3.f;
    static constexpr float most_l = 0x1p40f, way = 56.f, alone = 0x1p-7f;
};

template <typename T, int F, int DP, int MT>
struct CacheRowsCfg {
    using P = CacheProduct<T, F>;
    static constexpr int E = 16 / P::es;                  // channels a 16-byte chunk
    static constexpr int RB = DP * P::es, CH = RB / 16;   // bytes and chunks a row
    static constexpr int EV = DP / 8 < E ? DP / 8 : E;    // channels of V a lane has at a time
    static constexpr int KS = RB >= 256 ? 16 : 32;        // keys a step
    static constexpr int kStage = 2 * KS * RB;
    static constexpr int kStages = 3;
    static constexpr int kTailStage = 2 * 16 * DP * (int)sizeof(T);
    static constexpr int kRing = kStages * kStage > kTailStage ? kStages * kStage : kTailStage;
    static constexpr int kTailStages = F == kCacheSame ? kStages : kRing / kTailStage >= 2 ? 2 : 1;
    static constexpr int kTailKeys = F == kCacheSame ? KS : 16;
    static constexpr int kFragments = MT * (DP / 16) * 32 * 16;  // bytes of a piece of the queries
    static constexpr int kQ = kFragments * (P::qp + (F == kCacheSame ? 0 : CacheProduct<T, kCacheSame>::qp));
    static constexpr int kOut = kCacheWarps * MT * 16 * (DP + 4) * 4;  // the warps' parts, over the ring
    static constexpr int kSmem = kQ + (kCacheWarps * kRing > kOut ? kCacheWarps * kRing : kOut);
    static constexpr int kResident = kSmem > 111 * 1024 ? 1 : kSmem > 73 * 1024 ? 2 : 3;
};

__device__ __forceinline__ uint32_t cache_smem(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cache_copy16(uint32_t dst, const void* src, uint32_t bytes) {  // bytes: 16, or 0 for zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cache_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cache_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <bool BF16>
__device__ __forceinline__ void cache_mma(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
template <bool BF16>
__device__ __forceinline__ uint32_t cache_pack(float lo, float hi) {
    uint32_t r;
    if constexpr (BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <bool BF16>
__device__ __forceinline__ float2 cache_unpack(uint32_t v) {
    if constexpr (BF16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
// two values in N pieces of 16 bits, each what the ones before leave, rounded
template <bool BF16, int N>
__device__ __forceinline__ void cache_pieces(float lo, float hi, uint32_t (&p)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        p[i] = cache_pack<BF16>(lo, hi);
        if (i + 1 < N) {
            const float2 f = cache_unpack<BF16>(p[i]);
            lo -= f.x, hi -= f.y;
        }
    }
}
__device__ __forceinline__ float cache_ex2(float x) {  // 2 units in the last place; 0 for -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Where a row's 16-byte chunk lies in a stage (rows of RB bytes).  Both reads take eight lanes at a time: K two rows (2k, 2k + 1) of
// chunks 0..3 or 4..7, V four rows (all even or all odd) of two chunks that follow one another.
template <int RB>
__device__ __forceinline__ int cache_chunk(int row, int chunk) {
    if constexpr (RB == 64) {
        return (row >> 1) * 128 + (((((row & 1) << 2) | chunk) ^ (((row >> 1) & 3) << 1)) << 4);
    } else {
        const int f = (((row >> 1) & 3) << 1) ^ ((row & 1) << 2);
        return row * RB + ((chunk ^ f) << 4);  // f < 8: stays within the row's line of 128 bytes
    }
}

// The state of a warp's rows: MT tiles of 16, of each the rows lane / 4 and lane / 4 + 8.
template <int DP, int MT>
struct CacheState {
    float o[MT][DP / 8][4];
    float m[MT][2], l[MT][2];
    float low[MT][2], alone[MT][2];  // f16: a lane's sum that asks for a lower m (0: none), the largest key's part of the row's sum
    uint32_t top;  // 8 bits: O is in units of the scale of this byte (the largest met)
};
constexpr float kCacheNone = -1e30f;  // m before any score

// One walk over steps of KS keys: `cached` ones over the cache in format F, then `fresh` ones over the new tokens in the queries'
// type (one of the two is 0 where F is a format of codes).  E, EV: which channels a lane has, those of the cache's format in both.
template <typename T, int F, int DP, int MT, int E, int EV, int KS, int STAGES>
struct CacheWalk {
    using P = CacheProduct<T, F>;
    static constexpr int RB = DP * P::es, CH = RB / 16, EC = 16 / P::es, NT = KS / 8, GR = KS / 16, SETS = DP / (8 * EV);
    static constexpr int kStage = 2 * KS * RB;
    static constexpr bool kCodes = F != kCacheSame;

    const CacheArgs& a;
    const CacheUnit& u;
    unsigned char* ring;
    const uint4* qf;      // fragments [piece][MT][DP / 16][32]
    const float* factor;  // codes: [MT * 16], what scores of a row are multiplied by
    const int* token_of;  // [MT * 16]: a row's new token
    int lane, first, cached, first_new, fresh, step_keys;  // this warp's steps begin at keys first, first + step_keys, ...
    // pages of this warp's groups of 16 keys, 32 of them at a time in the lanes, and entries of the next 32
    int here, next, have;

    __device__ __forceinline__ int group_entry(int gi) const {
        const int token = first + (gi / GR) * step_keys + (gi % GR) * 16;
        return gi < cached * GR && token < u.length ? cache_entry(a.c, u.b, token) : kCacheNoPage;
    }

    // Starts the copies of step i, and reads the bytes of its scales (lane: key); which groups of 16 keys are there.
    // (The bytes stay untouched until their step comes: any arithmetic would wait for them here.)
    __device__ __forceinline__ void issue(int i, uint32_t& k_byte, uint32_t& v_byte, uint32_t& there) {
        const uint32_t dst = cache_smem(ring) + (uint32_t)(i % STAGES) * kStage;
        const int row0 = lane / CH, chunk = lane % CH;  // a row takes CH lanes, or each lane CH / 32 chunks of it
#pragma unroll 1
        for (int g = 0; g < GR; ++g) {
            const char *k, *v;
            long long kst, vst;
            int left;
            if (i < cached) {
                const int gi = i * GR + g, token = first + i * step_keys + g * 16;
                if (gi >= have + 32) {  // asked for in ascending order
                    have += 32;
                    here = cache_page_of(a.c, next);
                    next = group_entry(have + 32 + lane);
                }
                const int page = __shfl_sync(0xffffffffu, here, gi & 31);
                const long long p = max(page, 0);
                const int in_page = token & (a.c.page - 1);
                left = page < 0 ? 0 : u.length - token;
                if (page >= 0) there |= 1u << g;
                k = static_cast<const char*>(a.c.k) + (p * a.c.k_sp + in_page * a.c.k_st + u.n * a.c.k_sh) * P::es;
                v = static_cast<const char*>(a.c.v) + (p * a.c.v_sp + in_page * a.c.v_st + u.n * a.c.v_sh) * P::es;
                kst = a.c.k_st * P::es, vst = a.c.v_st * P::es;
                if constexpr (kCodes) {
                    const int row = lane - g * 16;
                    if ((unsigned)row < 16u && row < left) {
                        k_byte = a.c.ks[p * a.c.ks_sp + (in_page + row) * a.c.ks_st + u.n * a.c.ks_sh];
                        v_byte = a.c.vs[p * a.c.vs_sp + (in_page + row) * a.c.vs_st + u.n * a.c.vs_sh];
                    }
                }
            } else {
                const int j = first_new + (i - cached) * step_keys + g * 16;
                left = u.count - j;
                const long long at = left > 0 ? j : 0;
                k = reinterpret_cast<const char*>(static_cast<const T*>(a.nk) + u.b * a.nk_sb + at * a.nk_st + u.n * a.nk_sh);
                v = reinterpret_cast<const char*>(static_cast<const T*>(a.nv) + u.b * a.nv_sb + at * a.nv_st + u.n * a.nv_sh);
                kst = a.nk_st * P::es, vst = a.nv_st * P::es;
            }
            const char *k0 = k + row0 * kst, *v0 = v + row0 * vst;
#pragma unroll
            for (int x = 0; x < 16 * CH / 32; ++x) {
                constexpr int STEP = CH < 32 ? 32 / CH : 1;
                const int row = row0 + x * STEP;
                const bool in = row < left && chunk * EC < a.D;
                const uint32_t at = dst + cache_chunk<RB>(g * 16 + row, chunk);
                cache_copy16(at, in ? k0 + chunk * 16 : k, in ? 16 : 0);
                cache_copy16(at + KS * RB, in ? v0 + chunk * 16 : v, in ? 16 : 0);
                k0 += STEP * kst, v0 += STEP * vst;
            }
        }
    }

    // the four channels of key `row` that this lane has at K step s, as N-piece operands
    __device__ __forceinline__ void k_operand(const unsigned char* k, int row, int s, uint32_t (&b)[P::kp][2]) const {
        const int c = lane & 3, ch = E * (c + 4 * (s / (E / 4))) + 4 * (s % (E / 4));
        const unsigned char* at = k + cache_chunk<RB>(row, ch / EC) + (ch % EC) * P::es;
        if constexpr (P::es == 4) {
            const float4 x = *reinterpret_cast<const float4*>(at);
            uint32_t lo[3], hi[3];
            cache_pieces<true, 3>(x.x, x.y, lo);
            cache_pieces<true, 3>(x.z, x.w, hi);
#pragma unroll
            for (int i = 0; i < 3; ++i) b[i][0] = lo[i], b[i][1] = hi[i];
        } else if constexpr (P::es == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(at);
            b[0][0] = x.x, b[0][1] = x.y;
        } else {
            cache_four_f16<F>(*reinterpret_cast<const uint32_t*>(at), b[0][0], b[0][1]);
        }
    }

    __device__ __forceinline__ void scores(const unsigned char* k, float (&s)[MT][NT][4]) const {
        const int g = lane >> 2;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][j][e] = 0.f;
        constexpr int STEPS = DP / 16;
        if constexpr (E == EC && P::es < 4) {  // a 16-byte chunk at a time: E / 4 steps
#pragma unroll
            for (int i = 0; i < STEPS / (E / 4); ++i) {
                uint4 x[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    x[j] = *reinterpret_cast<const uint4*>(k + cache_chunk<RB>(j * 8 + g, (lane & 3) + 4 * i));
#pragma unroll
                for (int h = 0; h < E / 4; ++h) {
                    const int st = i * (E / 4) + h;
                    uint4 q[P::qp][MT];
#pragma unroll
                    for (int p = 0; p < P::qp; ++p)
#pragma unroll
                        for (int t = 0; t < MT; ++t) q[p][t] = qf[((p * MT + t) * STEPS + st) * 32 + lane];
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
                        uint32_t b0, b1;
                        if constexpr (P::es == 2) b0 = w[2 * h], b1 = w[2 * h + 1];
                        else cache_four_f16<F>(w[h], b0, b1);
#pragma unroll
                        for (int p = P::qp - 1; p >= 0; --p)
#pragma unroll
                            for (int t = 0; t < MT; ++t) cache_mma<P::bf16>(s[t][j], q[p][t], b0, b1);
                    }
                }
            }
        } else {
#pragma unroll
            for (int st = 0; st < STEPS; ++st) {
                uint4 q[P::qp][MT];
#pragma unroll
                for (int p = 0; p < P::qp; ++p)
#pragma unroll
                    for (int t = 0; t < MT; ++t) q[p][t] = qf[((p * MT + t) * STEPS + st) * 32 + lane];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    uint32_t b[P::kp][2];
                    k_operand(k, j * 8 + g, st, b);
#pragma unroll
                    for (int sum = P::kp == 1 ? P::qp - 1 : 2; sum >= 0; --sum)  // pieces x and y with x + y = sum: small products first
#pragma unroll
                        for (int x = sum; x >= 0; --x)
                            if (x < P::qp && sum - x < P::kp)
#pragma unroll
                                for (int t = 0; t < MT; ++t) cache_mma<P::bf16>(s[t][j], q[x][t], b[sum - x][0], b[sum - x][1]);
                }
            }
        }
    }

    // O += P V for the keys 16 kk .. 16 kk + 15
    __device__ __forceinline__ void outputs(const unsigned char* v, int kk, const uint4 (&p)[P::pp][MT], CacheState<DP, MT>& z) const {
        const int g = lane >> 2, c = lane & 3;
        constexpr int WORDS = EV * P::es / 4;
#pragma unroll
        for (int set = 0; set < SETS; ++set) {
            uint32_t w[4][WORDS];
            const int ch = E == EV ? E * (g + 8 * set) : EV * g;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = kk * 16 + 2 * c + (r & 1) + (r >> 1) * 8;
                if constexpr (WORDS == 2) {
                    const uint2 x = *reinterpret_cast<const uint2*>(v + cache_chunk<RB>(row, ch / EC) + (ch % EC) * P::es);
                    w[r][0] = x.x, w[r][1] = x.y;
                } else {
#pragma unroll
                    for (int i = 0; i < WORDS / 4; ++i) {
                        const uint4 x = *reinterpret_cast<const uint4*>(v + cache_chunk<RB>(row, ch / EC + i));
                        w[r][4 * i] = x.x, w[r][4 * i + 1] = x.y, w[r][4 * i + 2] = x.z, w[r][4 * i + 3] = x.w;
                    }
                }
            }
            if constexpr (P::es == 2) {
#pragma unroll
                for (int j = 0; j < EV; ++j) {
                    const int sel = (j & 1) ? 0x7632 : 0x5410;
                    const uint32_t b0 = __byte_perm(w[0][j / 2], w[1][j / 2], sel), b1 = __byte_perm(w[2][j / 2], w[3][j / 2], sel);
#pragma unroll
                    for (int t = 0; t < MT; ++t) cache_mma<P::bf16>(z.o[t][set * EV + j], p[0][t], b0, b1);
                }
            } else if constexpr (P::es == 1) {
#pragma unroll
                for (int j = 0; j < EV; j += 4) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // channels j + 2h and j + 2h + 1: key, next key, key, next key
                        const int sel = h ? 0x7362 : 0x5140;
                        uint32_t x0, x1, y0, y1;
                        cache_four_f16<F>(__byte_perm(w[0][j / 4], w[1][j / 4], sel), x0, x1);
                        cache_four_f16<F>(__byte_perm(w[2][j / 4], w[3][j / 4], sel), y0, y1);
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            if constexpr (P::f32) {  // a step's products start anew and are added in binary32, the small piece first
                                float d[2][4] = {};
#pragma unroll
                                for (int i = P::pp - 1; i >= 0; --i) {
                                    cache_mma<P::bf16>(d[0], p[i][t], x0, y0);
                                    cache_mma<P::bf16>(d[1], p[i][t], x1, y1);
                                }
#pragma unroll
                                for (int e = 0; e < 4; ++e) z.o[t][set * EV + j + 2 * h][e] += d[0][e], z.o[t][set * EV + j + 2 * h + 1][e] += d[1][e];
                            } else {
                                cache_mma<P::bf16>(z.o[t][set * EV + j + 2 * h], p[0][t], x0, y0);
                                cache_mma<P::bf16>(z.o[t][set * EV + j + 2 * h + 1], p[0][t], x1, y1);
                            }
                        }
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < EV; ++j) {
                    uint32_t b0[3], b1[3];
                    cache_pieces<true, 3>(__uint_as_float(w[0][j]), __uint_as_float(w[1][j]), b0);
                    cache_pieces<true, 3>(__uint_as_float(w[2][j]), __uint_as_float(w[3][j]), b1);
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        float d[4] = {0.f, 0.f, 0.f, 0.f};  // a step's products start anew and are added in binary32
#pragma unroll
                        for (int sum = 2; sum >= 0; --sum)
#pragma unroll
                            for (int x = sum; x >= 0; --x) cache_mma<true>(d, p[x][t], b0[sum - x], b1[sum - x]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) z.o[t][set * EV + j][e] += d[e];
                    }
                }
            }
        }
    }

    __device__ __forceinline__ void compute(int i, uint32_t k_byte, uint32_t v_byte, uint32_t there, CacheState<DP, MT>& z) {
        const unsigned char* k = ring + (i % STAGES) * kStage;
        const unsigned char* v = k + KS * RB;
        const int g = lane >> 2, c = lane & 3;
        float s[MT][NT][4];
        scores(k, s);
        float vs[NT][2];  // scales of the values of the keys 8 j + 2 c and the next
        if constexpr (kCodes) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, v_byte == 255u ? 0u : v_byte);
            if (top > z.top) {
                const float f = z.top + 126 < top ? 0.f : cache_scale(127 + z.top - top);
                z.top = top;
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int d = 0; d < DP / 8; ++d)
#pragma unroll
                        for (int e = 0; e < 4; ++e) z.o[t][d][e] *= f;
            }
            const uint32_t below = v_byte == 0u ? 0u : (uint32_t)max((int)(127u + v_byte - z.top), 0) & 255u;  // this lane's key
            const uint32_t bytes = k_byte | (below << 8), pair = bytes | (__shfl_down_sync(0xffffffffu, bytes, 1) << 16);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint32_t two = __shfl_sync(0xffffffffu, pair, j * 8 + 2 * c);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t y = e ? two >> 16 : two & 0xffffu;
                    const float ks = cache_scale(y & 255u);
                    vs[j][e] = cache_scale(y >> 8);
#pragma unroll
                    for (int t = 0; t < MT; ++t) s[t][j][e] *= ks, s[t][j][2 + e] *= ks;
                }
            }
            if (__builtin_expect(__any_sync(0xffffffffu, k_byte == 255u || v_byte == 255u), 0)) {  // rows that are NaN, whatever their codes
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t kb = __shfl_sync(0xffffffffu, k_byte, j * 8 + 2 * c + e), vb = __shfl_sync(0xffffffffu, v_byte, j * 8 + 2 * c + e);
                        vs[j][e] = vb == 255u ? cache_row_scale(255u) : vs[j][e];
#pragma unroll
                        for (int t = 0; t < MT; ++t)
#pragma unroll
                            for (int h = 0; h < 2; ++h) s[t][j][2 * h + e] = kb == 255u ? cache_row_scale(255u) : s[t][j][2 * h + e];
                    }
            }
        }
        if (i >= cached) {
            const int key0 = first_new + (i - cached) * step_keys;
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int q = token_of[t * 16 + g + 8 * h];
                    const uint8_t* mask = a.mask ? a.mask + u.b * a.mk_sb + q * a.mk_sq : nullptr;
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int key = key0 + j * 8 + 2 * c + e;
                            const bool on = key < u.count && q < u.count && (mask ? mask[key] != 0 : key <= q);
                            if (!on) s[t][j][2 * h + e] = -attn_inf();
                        }
                }
        } else {
            const int key0 = first + i * step_keys;
            if (key0 + KS > u.length || there != (1u << GR) - 1) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const bool on = key0 + j * 8 + 2 * c + e < u.length && ((there >> (j / 2)) & 1u);
#pragma unroll
                        for (int t = 0; t < MT; ++t)
                            if (!on) s[t][j][e] = s[t][j][2 + e] = -attn_inf();
                    }
            }
        }
        // P against the reference at hand, and once more where a sum asks for another (the first step's does)
        float f[MT][2], p[MT][NT][4], sum[MT][2];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) f[t][h] = kCodes ? factor[t * 16 + g + 8 * h] : a.c2;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
            bool renew = false;
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    sum[t][h] = 0.f;
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float x = cache_ex2(fmaf(s[t][j][2 * h + e], f[t][h], -z.m[t][h]));
                            p[t][j][2 * h + e] = x;
                            sum[t][h] += x;
                        }
                    renew |= !(sum[t][h] <= P::most && (P::bf16 || sum[t][h] >= z.low[t][h]));
                }
            if (pass > 0) {
                if constexpr (!P::bf16) {
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float all = z.l[t][h] + sum[t][h];
                            all += __shfl_xor_sync(0xffffffffu, all, 1);
                            all += __shfl_xor_sync(0xffffffffu, all, 2);
                            z.low[t][h] = all - z.alone[t][h] < z.alone[t][h] * P::alone && all < P::most_l ? P::low : 0.f;
                        }
                }
                break;
            }
            if (!__any_sync(0xffffffffu, renew)) break;
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float top = -attn_inf();
#pragma unroll
                    for (int j = 0; j < NT; ++j) top = fmaxf(top, fmaxf(s[t][j][2 * h], s[t][j][2 * h + 1]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    top *= f[t][h];
                    float m = fmaxf(z.m[t][h], top - P::below);
                    if constexpr (!P::bf16) {
                        if (m > z.m[t][h]) z.alone[t][h] = exp2f(P::below);
                        if (z.low[t][h] > 0.f && top < z.m[t][h] - P::drop && top > z.m[t][h] - P::way) m = top - P::below_low;
                    }
                    const float by = m == z.m[t][h] ? 1.f : cache_ex2(z.m[t][h] - m);
                    if (!P::bf16 && m < z.m[t][h]) z.alone[t][h] *= by;
                    z.m[t][h] = m;
                    z.l[t][h] *= by;
#pragma unroll
                    for (int d = 0; d < DP / 8; ++d) z.o[t][d][2 * h] *= by, z.o[t][d][2 * h + 1] *= by;
                }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) z.l[t][h] += sum[t][h];
#pragma unroll
        for (int kk = 0; kk < GR; ++kk) {
            uint4 pf[P::pp][MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                uint32_t x[4][P::pp];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float lo = p[t][2 * kk + (e >> 1)][2 * (e & 1)], hi = p[t][2 * kk + (e >> 1)][2 * (e & 1) + 1];
                    if constexpr (kCodes) lo *= vs[2 * kk + (e >> 1)][0], hi *= vs[2 * kk + (e >> 1)][1];
                    cache_pieces<P::bf16, P::pp>(lo, hi, x[e]);
                }
#pragma unroll
                for (int i2 = 0; i2 < P::pp; ++i2) pf[i2][t] = make_uint4(x[0][i2], x[1][i2], x[2][i2], x[3][i2]);
            }
            outputs(v, kk, pf, z);
        }
    }

    // `prepare`: what the block has to do before the first products, once its first copies are on their way.
    template <typename Prepare>
    __device__ __forceinline__ void run(CacheState<DP, MT>& z, Prepare prepare) {
        const int steps = cached + fresh;
        if (cached > 0) {
            here = group_entry(lane);
            next = group_entry(32 + lane);
            here = cache_page_of(a.c, here);
            have = 0;
        }
        uint32_t kb[STAGES], vb[STAGES], there[STAGES];  // of the steps in flight, the nearest first
#pragma unroll
        for (int j = 0; j < STAGES; ++j) kb[j] = vb[j] = there[j] = 0;
        // one place for the copies and one for the products, the copies STAGES - 1 steps ahead
#pragma unroll 1
        for (int i = 1 - STAGES; i < max(steps, 1); ++i) {
            if constexpr (STAGES > 1) {
                cache_wait<(STAGES > 1 ? STAGES - 2 : 0)>();
                __syncwarp();  // the step's copies of all lanes are there, and the stage of step i - 1 is read
            } else {
                __syncwarp();
            }
            kb[STAGES - 1] = vb[STAGES - 1] = there[STAGES - 1] = 0;
            if (i + STAGES - 1 < steps) issue(i + STAGES - 1, kb[STAGES - 1], vb[STAGES - 1], there[STAGES - 1]);
            cache_commit();
            if constexpr (STAGES == 1) {
                cache_wait<0>();
                __syncwarp();
            }
            if (i == 0) prepare();
            if (i >= 0 && i < steps) compute(i, kb[0], vb[0], there[0], z);
#pragma unroll
            for (int j = 0; j + 1 < STAGES; ++j) kb[j] = kb[j + 1], vb[j] = vb[j + 1], there[j] = there[j + 1];
        }
        cache_wait<0>();
        __syncwarp();
    }
};

template <typename T>
__device__ __forceinline__ void cache_four(const T* p, float (&y)[4]) {
    if constexpr (sizeof(T) == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        y[0] = x.x, y[1] = x.y, y[2] = x.z, y[3] = x.w;
    } else {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        const float2 lo = cache_unpack<CacheType<T>::code == 2>(x.x), hi = cache_unpack<CacheType<T>::code == 2>(x.y);
        y[0] = lo.x, y[1] = lo.y, y[2] = hi.x, y[3] = hi.y;
    }
}

template <typename T, int F, int DP, int MT>
__global__ void __launch_bounds__(kCacheWarps * 32, CacheRowsCfg<T, F, DP, MT>::kResident) msda_cache_rows_kernel(const CacheArgs a) {
    using Cfg = CacheRowsCfg<T, F, DP, MT>;
    using P = CacheProduct<T, F>;
    using PT = CacheProduct<T, kCacheSame>;
    using Ty = CacheType<T>;
    constexpr int R = MT * 16, STEPS = DP / 16, OB = DP + 4, KS = Cfg::KS, KT = Cfg::kTailKeys;
    constexpr bool CODES = F != kCacheSame;
    extern __shared__ __align__(128) unsigned char cache_smem_raw[];
    __shared__ CacheStart start;
    __shared__ float factor[R], up[R], part_m[kCacheWarps][R], part_l[kCacheWarps][R];
    __shared__ int token_of[R], head_of[R];  // of a row; token T: there is none
    uint4* qf = reinterpret_cast<uint4*>(cache_smem_raw);
    uint4* qt = CODES ? qf + P::qp * Cfg::kFragments / 16 : qf;
    unsigned char* ring = cache_smem_raw + Cfg::kQ;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    if (warp == 0) {
        const CacheStart s = cache_start(a);
        if (lane == 0) start = s;
    }
    __syncthreads();

    cache_walk(a, start, threadIdx.x == 0, [&](const CacheUnit& u, int tile, int tiles, int slot) {
        const T* query = static_cast<const T*>(a.q) + u.b * a.q_sb + (long long)u.n * a.G * a.q_sh;
        __syncthreads();  // the unit before is out
        if (threadIdx.x < R) {
            const int x = u.rt * R + threadIdx.x, t = x / a.G;
            token_of[threadIdx.x] = x < a.rows ? t : a.T;
            head_of[threadIdx.x] = x - t * a.G;
        }
        __syncthreads();
        auto prepare = [&] {
            // ---- codes: a power of two that brings a row's largest to 2^14 or more ----
            if constexpr (CODES) {
#pragma unroll 1
                for (int r = warp; r < R; r += kCacheWarps) {
                    const int t = token_of[r];
                    float top = 0.f;
                    if (t < u.count && lane * 4 < a.D) {
                        float y[4];
                        cache_four(query + t * a.q_st + head_of[r] * a.q_sh + lane * 4, y);
                        top = fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3])));
                    }
                    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
                    const int e = (int)(__float_as_uint(top) >> 23);  // 2^(e - 127) <= top
                    const float by = e > 0 && e < 255 ? __uint_as_float((uint32_t)min(268 - e, 227) << 23) : 1.f;
                    if (lane == 0) {
                        up[r] = by;
                        factor[r] = fmaxf(a.c2 * (1.f / by), 1e-37f);  // a power of two: exact; never 0, which would make NaN of what is hidden
                    }
                }
                __syncthreads();
            }
            // ---- the queries' fragments: entry (tile t of 16, step s, lane) are the channels of lane % 4 at step s of rows lane / 4 and + 8 ----
#pragma unroll 1
            for (int x = threadIdx.x; x < MT * STEPS * 32; x += kCacheWarps * 32) {
                const int ln = x & 31, s = (x >> 5) % STEPS, t = (x >> 5) / STEPS;
                const int ch = Cfg::E * ((ln & 3) + 4 * (s / (Cfg::E / 4))) + 4 * (s % (Cfg::E / 4));
                float y[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = t * 16 + (ln >> 2) + 8 * h, tok = token_of[r];
                    y[h][0] = y[h][1] = y[h][2] = y[h][3] = 0.f;
                    if (tok < u.count && ch < a.D) cache_four(query + tok * a.q_st + head_of[r] * a.q_sh + ch, y[h]);
                }
                auto put = [&](uint4* to, auto product, float up0, float up1) {
                    using Q = decltype(product);
                    uint32_t f[4][Q::qp];
                    cache_pieces<Q::bf16, Q::qp>(y[0][0] * up0, y[0][1] * up0, f[0]);
                    cache_pieces<Q::bf16, Q::qp>(y[1][0] * up1, y[1][1] * up1, f[1]);
                    cache_pieces<Q::bf16, Q::qp>(y[0][2] * up0, y[0][3] * up0, f[2]);
                    cache_pieces<Q::bf16, Q::qp>(y[1][2] * up1, y[1][3] * up1, f[3]);
#pragma unroll
                    for (int p = 0; p < Q::qp; ++p) to[((p * MT + t) * STEPS + s) * 32 + ln] = make_uint4(f[0][p], f[1][p], f[2][p], f[3][p]);
                };
                if constexpr (CODES) {
                    put(qf, P{}, up[t * 16 + (ln >> 2)], up[t * 16 + (ln >> 2) + 8]);
                    if (a.nk) put(qt, PT{}, 1.f, 1.f);
                } else {
                    put(qf, P{}, 1.f, 1.f);
                }
            }
            __syncthreads();
        };

        CacheState<DP, MT> z;
        z.top = 0;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
            for (int h = 0; h < 2; ++h) z.m[t][h] = kCacheNone, z.l[t][h] = z.low[t][h] = z.alone[t][h] = 0.f;
#pragma unroll
            for (int d = 0; d < DP / 8; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) z.o[t][d][e] = 0.f;
        }
        unsigned char* my_ring = ring + warp * Cfg::kRing;
        // this warp's steps over the cache, and over the new tokens
        constexpr int step = kCacheWarps * KS, step_new = kCacheWarps * KT;
        const int last = min(tile + tiles, u.cache_tiles), first = tile * step + warp * KS;
        const int cached = max(0, min(last - tile, (u.length - first + step - 1) / step));
        int fresh = 0, first_new = 0;
        if (a.nk && tile + tiles > u.cache_tiles) {
            const int at = max(0, tile - u.cache_tiles), end = min(cache_tail_keys(a, u.rt, u.count), (tile + tiles - u.cache_tiles) * step_new);
            first_new = at * step_new + warp * KT;
            fresh = first_new < end ? (end - first_new + step_new - 1) / step_new : 0;
        }
        if constexpr (CODES) {
            CacheWalk<T, F, DP, MT, Cfg::E, Cfg::EV, KS, Cfg::kStages> walk{a, u, my_ring, qf, factor, token_of, lane, first, cached, 0, 0, step, 0, 0, 0};
            walk.run(z, prepare);
            if (z.top != 0) {  // back to units of 1, with m where the largest key asks for it: a lower one makes large values infinite
                const float f = cache_scale(z.top);
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int e = max((int)(__float_as_uint(z.alone[t][h]) >> 23) - 127 - (int)P::below, 0);  // places that m went down
                        const float by = cache_scale(127 - e);
                        z.m[t][h] += e, z.l[t][h] *= by, z.alone[t][h] *= by;
#pragma unroll
                        for (int d = 0; d < DP / 8; ++d) z.o[t][d][2 * h] = z.o[t][d][2 * h] * by * f, z.o[t][d][2 * h + 1] = z.o[t][d][2 * h + 1] * by * f;
                    }
            }
            if (fresh > 0) {
                CacheWalk<T, kCacheSame, DP, MT, Cfg::E, Cfg::EV, KT, Cfg::kTailStages> walk{a, u, my_ring, qt, factor, token_of, lane, 0, 0, first_new, fresh, step_new, 0, 0, 0};
                walk.run(z, [] {});
            }
        } else {
            CacheWalk<T, F, DP, MT, Cfg::E, Cfg::EV, KS, Cfg::kStages> walk{a, u, my_ring, qf, factor, token_of, lane, first, cached, first_new, fresh, step, 0, 0, 0};
            walk.run(z, prepare);
        }
        __syncthreads();  // rings are done with
        // ---- the warps' parts, joined in their order ----
        float* po = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = t * 16 + g + 8 * h;
                float l = z.l[t][h];
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                if (c == 0) part_m[warp][r] = z.m[t][h], part_l[warp][r] = l;
#pragma unroll
                for (int d = 0; d < DP / 8; ++d)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int set = d / Cfg::EV, j = d % Cfg::EV, lane8 = 2 * c + e;
                        const int ch = (Cfg::E == Cfg::EV ? Cfg::E * (lane8 + 8 * set) : Cfg::EV * lane8) + j;
                        po[(warp * R + r) * OB + ch] = z.o[t][d][2 * h + e];
                    }
            }
        __syncthreads();
#pragma unroll 1
        for (int x = threadIdx.x; x < R * (DP / 4); x += kCacheWarps * 32) {
            const int r = x / (DP / 4), d = x % (DP / 4) * 4, t = token_of[r];
            if (t >= a.T || d >= a.D) continue;
            float top = kCacheNone;
#pragma unroll
            for (int w = 0; w < kCacheWarps; ++w) top = fmaxf(top, part_m[w][r]);
            float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kCacheWarps; ++w) {
                const float f = exp2f(part_m[w][r] - top);
                sum += part_l[w][r] * f;
                const float4 y = *reinterpret_cast<const float4*>(&po[(w * R + r) * OB + d]);
                o[0] += y.x * f, o[1] += y.y * f, o[2] += y.z * f, o[3] += y.w * f;
            }
            const int h = u.n * a.G + head_of[r];
            const bool none = sum == 0.f || t >= u.count;
            const float l2 = none ? -attn_inf() : top + log2f(sum), inv = none ? 0.f : 1.f / sum;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = none ? 0.f : o[e] * inv;
            if (slot >= 0) {
                const long long at = (long long)slot * R + r;
                *reinterpret_cast<float4*>(a.part_o + at * a.D + d) = make_float4(o[0], o[1], o[2], o[3]);
                if (d == 0) a.part_l2[at] = l2;
            } else {
                T* out = static_cast<T*>(a.out) + (((long long)u.b * a.T + t) * a.M + h) * a.D + d;
#pragma unroll
                for (int e = 0; e < 4; ++e) out[e] = Ty::put(o[e]);
                if (d == 0) a.lse[((long long)u.b * a.M + h) * a.T + t] = l2 * kLn2;
            }
        }
    });
}

template <typename T, int F, int DP, int MT>
static CacheRowsShape cache_rows_shape_of() {
    using Cfg = CacheRowsCfg<T, F, DP, MT>;
    return {MT * 16, kCacheWarps * Cfg::KS, kCacheWarps * Cfg::kTailKeys, Cfg::kResident};
}
template <typename T, int F, int DP, int MT>
static cudaError_t cache_rows_go(const CacheArgs& a, int grid, cudaStream_t st) {
    using Cfg = CacheRowsCfg<T, F, DP, MT>;
    static SmemSeen seen;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(&msda_cache_rows_kernel<T, F, DP, MT>), Cfg::kSmem, seen);
    if (e != cudaSuccess) return e;
    msda_cache_rows_kernel<T, F, DP, MT><<<grid, kCacheWarps * 32, Cfg::kSmem, st>>>(a);
    return cudaGetLastError();
}

// Tiles of 32 rows only in binary32 up to 64 channels: 16 bits have the tensor-core kernel there, wider rows no registers.
#define MSDA_CACHE_ROWS_BY(format, D, rows, f, ...)                                                      \
    do {                                                                                                 \
        if constexpr (sizeof(T) == 4) {                                                                  \
            if ((rows) > 16 && (D) <= 64) {                                                              \
                if ((format) == kCacheSame) return f<T, kCacheSame, 64, 2>(__VA_ARGS__);                 \
                if ((format) == kCacheE4m3) return f<T, kCacheE4m3, 64, 2>(__VA_ARGS__);                 \
                return f<T, kCacheInt8, 64, 2>(__VA_ARGS__);                                             \
            }                                                                                            \
        }                                                                                                \
        if ((D) <= 64) {                                                                                 \
            if ((format) == kCacheSame) return f<T, kCacheSame, 64, 1>(__VA_ARGS__);                     \
            if ((format) == kCacheE4m3) return f<T, kCacheE4m3, 64, 1>(__VA_ARGS__);                     \
            return f<T, kCacheInt8, 64, 1>(__VA_ARGS__);                                                 \
        }                                                                                                \
        if ((format) == kCacheSame) return f<T, kCacheSame, 128, 1>(__VA_ARGS__);                        \
        if ((format) == kCacheE4m3) return f<T, kCacheE4m3, 128, 1>(__VA_ARGS__);                        \
        return f<T, kCacheInt8, 128, 1>(__VA_ARGS__);                                                    \
    } while (0)

template <typename T>
CacheRowsShape cache_rows_shape(int format, int D, int rows) {
    MSDA_CACHE_ROWS_BY(format, D, rows, cache_rows_shape_of);
}
template <typename T>
cudaError_t launch_cache_rows(const CacheArgs& a, int format, int grid, cudaStream_t st) {
    MSDA_CACHE_ROWS_BY(format, a.D, a.rows, cache_rows_go, a, grid, st);
}

}  // namespace msda
