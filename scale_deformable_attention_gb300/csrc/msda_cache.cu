// msda_cache.cu -- the paged cache of keys and values: checks and launches of
// msda_cache_write / _read / _attention, the kernels that write and read rows,
// and the one that joins the parts of units which several blocks shared.
//
// Reading is bound by memory, a quantised write by its arithmetic: a row of D channels lies in the lanes
// that 16 bytes of the unquantised type each make, so its largest magnitude takes
// log2(lanes) exchanges and every access is a whole vector.  A warp takes 16
// tokens of a head, so that pages, places and scales are looked up once for them
// by one lane each and handed on by shuffles; a block's warps take the heads of the
// same tokens.  The cache's side (head by head) is then read or written in runs of
// 16 rows, the other side in whole tokens.  8 x 22223 tokens of 8 heads of 64, e4m3 to bf16: 86 us, 88 % of the copy rate,
// bf16 97 us, 99 %; lookups in every lane took 132 us (ALU 51 % busy with addresses).  Prompts of 8 x up to 16641 tokens of 4
// heads of 128 written: bf16 47 us, 91 %; to e4m3 55 us, 59 % (ALU 52 %: largest of a row, scale, codes).  Four blocks an SM in
// 16 bits (three: 97 us), three in binary32 (four: 29 us against 27 for 4 x 8191 tokens of 8 heads of 48).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <limits>
#include <type_traits>

#include "msda_attention_tc.cuh"
#include "msda_cache.cuh"
#include "msda_cache_tc.cuh"
#include "msda_host.cuh"

namespace msda {

namespace {

constexpr int kMoveThreads = 256;

template <typename T>
struct CacheVec;
template <>
struct CacheVec<float> {
    static __device__ __forceinline__ float most() { return __uint_as_float(0x7f7fffffu); }  // the largest finite value
    static constexpr int n = 4;
    static __device__ __forceinline__ void get(const uint4& x, float (&v)[4]) {
        v[0] = __uint_as_float(x.x), v[1] = __uint_as_float(x.y), v[2] = __uint_as_float(x.z), v[3] = __uint_as_float(x.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};
template <>
struct CacheVec<__half> {
    static __device__ __forceinline__ float most() { return __uint_as_float(0x477fe000u); }  // the largest finite value
    static constexpr int n = 8;
    static __device__ __forceinline__ void get(const uint4& x, float (&v)[8]) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&v)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct CacheVec<__nv_bfloat16> {
    static __device__ __forceinline__ float most() { return __uint_as_float(0x7f7f0000u); }  // the largest finite value
    static constexpr int n = 8;
    static __device__ __forceinline__ void get(const uint4& x, float (&v)[8]) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    static __device__ __forceinline__ uint4 put(const float (&v)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// A row's scale from its largest magnitude: the least power of two, 2^(byte - 127), that brings it into the codes' range
// (448 = 7/8 2^9, 127 = 127/128 2^7); 2^-100 at least.
template <int F>
__device__ __forceinline__ uint32_t cache_scale_byte(float top) {
    const uint32_t bits = __float_as_uint(top), e = bits >> 23, m = bits & 0x7fffffu;  // top = 1.m 2^(e - 127)
    if (e == 255u) return 255u;
    constexpr uint32_t most = F == kCacheE4m3 ? 0x600000u : 0x7e0000u;  // fraction bits of 1.75 and of 127/64
    constexpr int places = F == kCacheE4m3 ? 8 : 6;
    const int byte = (int)e - places + (m > most ? 1 : 0);
    return (uint32_t)max(byte, 27);
}
template <int F>
__device__ __forceinline__ uint32_t cache_codes(float a, float b, float c, float d) {
    if constexpr (F == kCacheE4m3) {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
        return (uint32_t)lo | ((uint32_t)hi << 16);
    } else {
        return ((uint32_t)__float2int_rn(a) & 255u) | (((uint32_t)__float2int_rn(b) & 255u) << 8) |
               (((uint32_t)__float2int_rn(c) & 255u) << 16) | ((uint32_t)__float2int_rn(d) << 24);
    }
}

}  // namespace

struct CacheMoveArgs {
    CachePages c;
    const void *key, *value;  // write: [B, source, N, D] at strides; read: outputs [B, T, N, D]
    long long k_sb, k_st, k_sh, v_sb, v_st, v_sh;
    const int *first, *counts, *select;  // write: start, counts or null, select [B, T] or null; read: lengths
    long long select_sb;
    int B, T, N, D, source;
    int lanes_log2;           // lanes a row: a power of two
};

constexpr int kMoveTokens = 16;

// A warp takes 16 tokens of one head, 32 / lanes rows at a time; a block's warps take the heads of the same tokens.  False where
// there are no such tokens.
__device__ __forceinline__ bool cache_piece(const CacheMoveArgs& a, int* t0, int* n) {
    const unsigned w = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5), block = w / (unsigned)a.N;
    *n = (int)(w - block * (unsigned)a.N);
    *t0 = (int)block * kMoveTokens;
    return *t0 < a.T;
}

// largest magnitude of a vector's elements as bits in the order of their size (NaN above infinity): of 16-bit types two maxima side by side
template <typename T>
__device__ __forceinline__ uint32_t cache_top(uint32_t a, uint32_t b) {
    if constexpr (sizeof(T) == 4) return max(a, b);
    else return __vmaxu2(a, b);
}
template <typename T>
__device__ __forceinline__ uint32_t cache_top(const uint4& x) {
    constexpr uint32_t m = sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu;
    return cache_top<T>(cache_top<T>(x.x & m, x.y & m), cache_top<T>(x.z & m, x.w & m));
}
template <typename T>
__device__ __forceinline__ float cache_top_value(uint32_t top) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(top);
    else {
        const uint32_t h = max(top & 0xffffu, top >> 16);
        if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half((unsigned short)h));
        else return __uint_as_float(h << 16);
    }
}

// x brought into -most..most; NaN stays NaN (a code of another program's may be one).
__device__ __forceinline__ float cache_clamp(float x, float most) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(-most));
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(most));
    return x;
}

// U rows of K and of V at a time a lane.
template <typename T, int F>
__global__ void __launch_bounds__(kMoveThreads, sizeof(T) == 4 ? 3 : 4) msda_cache_write_kernel(const CacheMoveArgs a) {
    constexpr int E = CacheVec<T>::n, U = 2, ES = F == kCacheSame ? (int)sizeof(T) : 1;
    const int lane = threadIdx.x & 31, at = lane & ((1 << a.lanes_log2) - 1), row0 = lane >> a.lanes_log2, rows = 32 >> a.lanes_log2;
    const bool in = at * E < a.D;
    int t0, n;
    if (!cache_piece(a, &t0, &n)) return;
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        const int count = cache_count(a.c, a.counts, b, a.T);
        if (t0 >= count) continue;
        // lane i < 16: where row t0 + i comes from and goes to (page -1: nowhere)
        int page = -1, place = 0, src = t0 + lane;
        if (lane < kMoveTokens && t0 + lane < count) {
            const long long token = (long long)a.first[b] + t0 + lane;
            if (token >= 0 && token < a.c.longest) {
                page = cache_page(a.c, b, (int)token);
                place = (int)token & (a.c.page - 1);
            } else {
                atomicOr(a.c.err, kCacheBad);
            }
            if (a.select) {
                src = a.select[b * a.select_sb + t0 + lane];
                if ((unsigned)src >= (unsigned)a.source) {
                    atomicOr(a.c.err, kCacheBad);
                    page = -1;
                }
            }
        }
        const T* key = static_cast<const T*>(a.key) + b * a.k_sb + n * a.k_sh + at * E;
        const T* value = static_cast<const T*>(a.value) + b * a.v_sb + n * a.v_sh + at * E;
        char* to_k = static_cast<char*>(a.c.k) + (n * a.c.k_sh + at * E) * ES;
        char* to_v = static_cast<char*>(a.c.v) + (n * a.c.v_sh + at * E) * ES;
        for (int r0 = 0; r0 < kMoveTokens && t0 + r0 < count; r0 += rows * U) {
            uint4 x[U][2];
            int pg[U], pl[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int r = r0 + i * rows + row0;
                pg[i] = __shfl_sync(0xffffffffu, page, r & 31);
                pl[i] = __shfl_sync(0xffffffffu, place, r & 31);
                const int from = __shfl_sync(0xffffffffu, src, r & 31);
                if (r >= kMoveTokens) pg[i] = -1;
                x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
                if (pg[i] >= 0 && in) {
                    x[i][0] = *reinterpret_cast<const uint4*>(key + from * a.k_st);
                    x[i][1] = *reinterpret_cast<const uint4*>(value + from * a.v_st);
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    char* to = w ? to_v + (pg[i] * a.c.v_sp + pl[i] * a.c.v_st) * ES : to_k + (pg[i] * a.c.k_sp + pl[i] * a.c.k_st) * ES;
                    if constexpr (F == kCacheSame) {
                        if (pg[i] >= 0 && in) *reinterpret_cast<uint4*>(to) = x[i][w];
                    } else {
                        uint32_t top = cache_top<T>(x[i][w]);
                        for (int l = a.lanes_log2 - 1; l >= 0; --l) top = cache_top<T>(top, __shfl_xor_sync(0xffffffffu, top, 1 << l));
                        const uint32_t byte = cache_scale_byte<F>(cache_top_value<T>(top));
                        const float up = __uint_as_float((254u - byte) << 23);
                        float v[E];
                        CacheVec<T>::get(x[i][w], v);
                        uint32_t codes[E / 4];
#pragma unroll
                        for (int e = 0; e < E / 4; ++e)
                            codes[e] = byte == 255u ? 0u : cache_codes<F>(v[4 * e] * up, v[4 * e + 1] * up, v[4 * e + 2] * up, v[4 * e + 3] * up);
                        if (pg[i] >= 0) {
                            if (in) {
                                if constexpr (E == 8) *reinterpret_cast<uint2*>(to) = make_uint2(codes[0], codes[1]);
                                else *reinterpret_cast<uint32_t*>(to) = codes[0];
                            }
                            if (at == 0) {
                                if (w) a.c.vs[pg[i] * a.c.vs_sp + pl[i] * a.c.vs_st + n * a.c.vs_sh] = (uint8_t)byte;
                                else a.c.ks[pg[i] * a.c.ks_sp + pl[i] * a.c.ks_st + n * a.c.ks_sh] = (uint8_t)byte;
                            }
                        }
                    }
                }
        }
    }
}

template <typename T, int F>
__global__ void __launch_bounds__(kMoveThreads, sizeof(T) == 4 ? 3 : 4) msda_cache_read_kernel(const CacheMoveArgs a) {
    constexpr int E = CacheVec<T>::n, U = 4, ES = F == kCacheSame ? (int)sizeof(T) : 1;
    const int lane = threadIdx.x & 31, at = lane & ((1 << a.lanes_log2) - 1), row0 = lane >> a.lanes_log2, rows = 32 >> a.lanes_log2;
    const bool in = at * E < a.D;
    int t0, n;
    if (!cache_piece(a, &t0, &n)) return;
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        const int here = min(kMoveTokens, a.T - t0);
        int left = min(here, cache_length(a.c, a.first, b) - t0);  // rows that the sequence has; the 16 tokens share a page
        const int page = left > 0 ? cache_page(a.c, b, t0) : -1, place = t0 & (a.c.page - 1);
        if (page < 0) left = 0;
        uint32_t bytes = 0;  // lane i < 16: row i's of K, lane 16 + i: of V
        if constexpr (F != kCacheSame) {
            const int r = lane & 15;
            if (r < left)
                bytes = lane < 16 ? a.c.ks[page * a.c.ks_sp + (place + r) * a.c.ks_st + n * a.c.ks_sh]
                                  : a.c.vs[page * a.c.vs_sp + (place + r) * a.c.vs_st + n * a.c.vs_sh];
        }
        const char* from_k = static_cast<const char*>(a.c.k) + (page * a.c.k_sp + place * a.c.k_st + n * a.c.k_sh + at * E) * ES;
        const char* from_v = static_cast<const char*>(a.c.v) + (page * a.c.v_sp + place * a.c.v_st + n * a.c.v_sh + at * E) * ES;
        const long long out = (((long long)b * a.T + t0) * a.N + n) * a.D + at * E;
        for (int r0 = 0; r0 < here; r0 += rows * U) {
            uint4 x[U][2];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int r = r0 + i * rows + row0;
                x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
                if (r < left && in) {
                    const char *k = from_k + r * a.c.k_st * ES, *v = from_v + r * a.c.v_st * ES;
                    if constexpr (F == kCacheSame) {
                        x[i][0] = *reinterpret_cast<const uint4*>(k), x[i][1] = *reinterpret_cast<const uint4*>(v);
                    } else if constexpr (E == 8) {
                        const uint2 p = *reinterpret_cast<const uint2*>(k), q = *reinterpret_cast<const uint2*>(v);
                        x[i][0].x = p.x, x[i][0].y = p.y, x[i][1].x = q.x, x[i][1].y = q.y;
                    } else {
                        x[i][0].x = *reinterpret_cast<const uint32_t*>(k), x[i][1].x = *reinterpret_cast<const uint32_t*>(v);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int r = r0 + i * rows + row0;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    uint4 y = x[i][w];
                    if constexpr (F != kCacheSame) {
                        const uint32_t byte = __shfl_sync(0xffffffffu, bytes, (r & 15) + 16 * w), c[2] = {y.x, y.y};
                        const float s = cache_row_scale(byte);
                        float v[E];
#pragma unroll
                        for (int e = 0; e < E / 4; ++e) {
                            uint32_t lo, hi;
                            cache_four_f16<F>(c[e], lo, hi);
                            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&lo)), q = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                            v[4 * e] = p.x * s, v[4 * e + 1] = p.y * s, v[4 * e + 2] = q.x * s, v[4 * e + 3] = q.y * s;
                        }
                        if (s * 512.f > CacheVec<T>::most()) {  // a code may be rounded up past the type's range: finite rows stay finite
#pragma unroll
                            for (int e = 0; e < E; ++e) v[e] = cache_clamp(v[e], CacheVec<T>::most());
                        }
                        y = CacheVec<T>::put(v);
                    }
                    if (r < here && in) *reinterpret_cast<uint4*>(static_cast<T*>(const_cast<void*>(w ? a.value : a.key)) + out + (long long)r * a.N * a.D) = y;
                }
            }
        }
    }
}

// Parts of the blocks that shared a unit: a block of 16 warps takes 16 rows of it, as many warps a row as there are (16 for one row, one
// for 16), each every so many-th part, a lane four channels; the warps of a row are joined in their order.  (Blocks cost more than
// what they do: one a row took 15 us, cold, for 8192 rows of two or three parts of 128 channels; four rows one after the other by four
// warps 5 us more for 16 units of 29 parts.)
constexpr int kJoinWarps = 16;
template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32) msda_cache_join_kernel(const CacheArgs a) {
    __shared__ float4 part[kJoinWarps][32];
    __shared__ float tops[kJoinWarps], sums[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // launched as a programmatic dependent of the kernel that makes the parts
    const int2 parts = a.units[blockIdx.x];
    if (parts.x < 0) return;
    int id = blockIdx.x;
    const int rt = id % a.row_tiles;
    id /= a.row_tiles;
    const int n = id % a.N, b = id / a.N, r0 = blockIdx.y * kJoinWarps;
    const int rows = min(kJoinWarps, min(a.tile_rows, a.rows - rt * a.tile_rows) - r0);  // of this block
    int each_log2 = 4;                                                                  // warps a row: a power of two
    while (each_log2 > 0 && (rows << each_log2) > kJoinWarps) --each_log2;
    const int each = 1 << each_log2, r = r0 + (warp >> each_log2), row = rt * a.tile_rows + r, mine = warp & (each - 1);
    const bool there = r - r0 < rows;
    float top = -attn_inf(), sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    // joins (l2, s, y) to (top, sum, o); NaN statistics make the row NaN
    auto join = [&](float l2, float s, const float4& y) {
        const float next = fmaxf(top, l2), ref = next == -attn_inf() ? 0.f : next, f = exp2f(top - ref), w = exp2f(l2 - ref);
        top = next, sum = sum * f + w * s;
        o[0] = o[0] * f + w * y.x, o[1] = o[1] * f + w * y.y, o[2] = o[2] * f + w * y.z, o[3] = o[3] * f + w * y.w;
    };
#pragma unroll 4
    for (int i = there ? mine : parts.y; i < parts.y; i += each) {
        // the first block's slot, then the first slots of the blocks behind it
        const long long at = (long long)(i == 0 ? parts.x : 2 * ((parts.x >> 1) + i)) * a.tile_rows + r;
        const float l2 = a.part_l2[at];
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (lane * 4 < a.D) y = *reinterpret_cast<const float4*>(a.part_o + at * a.D + lane * 4);
        join(l2, 1.f, y);
    }
    part[warp][lane] = make_float4(o[0], o[1], o[2], o[3]);
    if (lane == 0) tops[warp] = top, sums[warp] = sum;
    __syncthreads();
    if (!there || mine != 0) return;
    for (int w = 1; w < each; ++w) join(tops[warp + w], sums[warp + w], part[warp + w][lane]);
    const int t = row / a.G, h = n * a.G + row - t * a.G;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (lane * 4 < a.D) {
        T* out = static_cast<T*>(a.out) + (((long long)b * a.T + t) * a.M + h) * a.D + lane * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float y = sum == 0.f ? 0.f : o[e] * inv;
            if constexpr (sizeof(T) == 4) out[e] = y;
            else if constexpr (std::is_same<T, __half>::value) out[e] = __float2half_rn(y);
            else out[e] = __float2bfloat16_rn(y);
        }
    }
    if (lane == 0) a.lse[((long long)b * a.M + h) * a.T + t] = sum == 0.f ? -attn_inf() : ((top == -attn_inf() ? 0.f : top) + log2f(sum)) * kLn2;
}

template <typename T>
static cudaError_t join_go(const CacheArgs& a, bool early, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.B * a.N * a.row_tiles), (unsigned)(((a.rows < a.tile_rows ? a.rows : a.tile_rows) + kJoinWarps - 1) / kJoinWarps));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, &msda_cache_join_kernel<T>, a);
}
cudaError_t launch_cache_join(const CacheArgs& a, int dtype, bool early, cudaStream_t st) {
    return dtype == MSDA_F32 ? join_go<float>(a, early, st) : dtype == MSDA_F16 ? join_go<__half>(a, early, st) : join_go<__nv_bfloat16>(a, early, st);
}

}  // namespace msda

namespace {

using msda::CacheArgs;
using msda::CacheMoveArgs;
using msda::failf;

constexpr int64_t kMost = 1ll << 30;

bool positive(const int64_t* s) { return s[0] >= 0 && s[1] >= 0 && s[2] >= 0; }

// Tokens that a sequence has at most: none where there are no pages, whatever its length says (the kernels bring lengths into this
// range, raise the error bit and look at no table).
int64_t longest_of(const msda_cache_problem* p) { return p->pages > 0 ? p->longest : 0; }

// Sizes that all three calls share.
msda_status check(msda_dtype dt, int format, const msda_cache_problem* p) {
    if (dt != MSDA_F32 && dt != MSDA_F16 && dt != MSDA_BF16) return failf(MSDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
    if (format < MSDA_CACHE_SAME || format > MSDA_CACHE_INT8) return failf(MSDA_ERR_INVALID_ARG, "unknown cache format %d", format);
    if (!p) return failf(MSDA_ERR_INVALID_ARG, "problem is NULL");
    if (p->B < 0 || p->T < 0 || p->source < 0 || p->pages < 0 || p->width < 0 || p->longest < 0)
        return failf(MSDA_ERR_INVALID_ARG, "negative size (B=%lld T=%lld source=%lld pages=%lld width=%lld longest=%lld)", (long long)p->B,
                     (long long)p->T, (long long)p->source, (long long)p->pages, (long long)p->width, (long long)p->longest);
    if (p->N < 1 || p->D < 1) return failf(MSDA_ERR_INVALID_ARG, "N=%lld and D=%lld must be at least 1", (long long)p->N, (long long)p->D);
    if (p->D % 16 || p->D > msda::kAttnMaxChannels)
        return failf(MSDA_ERR_UNSUPPORTED, "D=%lld: the cache holds rows of 16, 32, ... %d channels", (long long)p->D, msda::kAttnMaxChannels);
    if (p->page < 16 || p->page > kMost || (p->page & (p->page - 1)))
        return failf(MSDA_ERR_UNSUPPORTED, "page=%lld must be a power of two of 16 or more", (long long)p->page);
    if (p->B > kMost || p->T > kMost || p->source > kMost || p->N > 65535 || p->pages > kMost || p->width > kMost || p->width * p->page > kMost)
        return failf(MSDA_ERR_UNSUPPORTED, "B=%lld, T=%lld, N=%lld, pages=%lld or width * page=%lld too large", (long long)p->B,
                     (long long)p->T, (long long)p->N, (long long)p->pages, (long long)(p->width > kMost ? p->width : p->width * p->page));
    if (p->longest > p->width * p->page)
        return failf(MSDA_ERR_INVALID_ARG, "longest=%lld above the table's %lld tokens", (long long)p->longest, (long long)(p->width * p->page));
    if (!positive(p->cache_key_stride) || !positive(p->cache_value_stride) || !positive(p->key_scale_stride) ||
        !positive(p->value_scale_stride) || !positive(p->query_stride) || !positive(p->key_stride) || !positive(p->value_stride) ||
        p->table_stride < 0 || p->mask_stride[0] < 0 || p->mask_stride[1] < 0 || p->select_stride < 0)
        return failf(MSDA_ERR_INVALID_ARG, "negative stride");
    return MSDA_OK;
}

// Rows of whole 16-byte vectors of elements of `es` bytes: the address, and the strides of dimensions of more than one.
msda_status vectors(const void* x, const int64_t* stride, int64_t a, int64_t b, int64_t c, size_t es, bool needed, const char* name) {
    if (!needed) return MSDA_OK;
    if (!x) return failf(MSDA_ERR_INVALID_ARG, "%s is NULL", name);
    const int64_t n[3] = {a, b, c};
    bool ok = msda::aligned_to(x, 16);
    for (int i = 0; i < 3; ++i) ok = ok && (n[i] <= 1 || (stride[i] * (int64_t)es) % 16 == 0);
    return ok ? MSDA_OK : failf(MSDA_ERR_MISALIGNED, "%s: rows must begin at multiples of 16 bytes", name);
}

msda_status cache_ok(msda_dtype dt, int format, const msda_cache_problem* p, const void* key, const void* value, const void* ks,
                     const void* vs, const int32_t* table, bool needed) {
    const size_t es = format != MSDA_CACHE_SAME ? 1 : dt == MSDA_F32 ? 4 : 2;
    const bool quantised = format != MSDA_CACHE_SAME;
    msda_status s;
    if ((s = vectors(key, p->cache_key_stride, p->pages, p->page, p->N, es, needed, "cache key")) ||
        (s = vectors(value, p->cache_value_stride, p->pages, p->page, p->N, es, needed, "cache value")) ||
        (s = msda::need_ptr(ks, needed && quantised, 1, "key scale")) || (s = msda::need_ptr(vs, needed && quantised, 1, "value scale")) ||
        (s = msda::need_ptr(table, needed, 4, "table")))
        return s;
    return MSDA_OK;
}

void three(const int64_t* s, long long& a, long long& b, long long& c) { a = s[0], b = s[1], c = s[2]; }

msda::CachePages pages_of(const msda_cache_problem* p, const void* key, const void* value, const void* ks, const void* vs, const int32_t* table) {
    msda::CachePages c{};
    c.k = const_cast<void*>(key), c.v = const_cast<void*>(value);
    c.ks = static_cast<uint8_t*>(const_cast<void*>(ks)), c.vs = static_cast<uint8_t*>(const_cast<void*>(vs));
    three(p->cache_key_stride, c.k_sp, c.k_st, c.k_sh);
    three(p->cache_value_stride, c.v_sp, c.v_st, c.v_sh);
    three(p->key_scale_stride, c.ks_sp, c.ks_st, c.ks_sh);
    three(p->value_scale_stride, c.vs_sp, c.vs_st, c.vs_sh);
    c.table = table, c.table_sb = p->table_stride;
    c.pages = (int)p->pages, c.page = (int)p->page, c.longest = (int)longest_of(p);
    while ((1 << c.page_log2) < c.page) ++c.page_log2;
    return c;
}

msda_status launched(cudaError_t e, const char* what) {
    return e == cudaSuccess ? MSDA_OK : failf(MSDA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

template <typename T, int F>
cudaError_t move_go(const CacheMoveArgs& a, bool write, dim3 grid, cudaStream_t st) {
    if (write) msda::msda_cache_write_kernel<T, F><<<grid, msda::kMoveThreads, 0, st>>>(a);
    else msda::msda_cache_read_kernel<T, F><<<grid, msda::kMoveThreads, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename T>
cudaError_t move_by_format(int format, CacheMoveArgs& a, bool write, cudaStream_t st) {
    const int vec = 16 / (int)sizeof(T);
    a.lanes_log2 = 1;
    while ((vec << a.lanes_log2) < a.D) ++a.lanes_log2;
    const long long pieces = ((long long)a.T + msda::kMoveTokens - 1) / msda::kMoveTokens * a.N, each = msda::kMoveThreads / 32;
    const dim3 grid((unsigned)((pieces + each - 1) / each), (unsigned)(a.B < 65535 ? a.B : 65535));
    if (format == MSDA_CACHE_SAME) return move_go<T, msda::kCacheSame>(a, write, grid, st);
    if (format == MSDA_CACHE_E4M3) return move_go<T, msda::kCacheE4m3>(a, write, grid, st);
    return move_go<T, msda::kCacheInt8>(a, write, grid, st);
}
msda_status move(msda_dtype dt, int format, CacheMoveArgs& a, bool write, cudaStream_t st) {
    msda_status s = msda::error_word(&a.c.err);
    if (s != MSDA_OK) return s;
    msda::TraceSpan ts(st);
    const cudaError_t e = dt == MSDA_F32   ? move_by_format<float>(format, a, write, st)
                          : dt == MSDA_F16 ? move_by_format<__half>(format, a, write, st)
                                           : move_by_format<__nv_bfloat16>(format, a, write, st);
    ts.end(write ? MSDA_KERNEL_CACHE_WRITE : MSDA_KERNEL_CACHE_READ, (int64_t)a.B * a.T * a.N);
    return launched(e, write ? "cache write kernel launch" : "cache read kernel launch");
}
// rows of one sequence are counted in 32 bits
msda_status move_size(const msda_cache_problem* p) {
    if ((p->T + 15) * p->N > 0x7fffffffll) return failf(MSDA_ERR_UNSUPPORTED, "T=%lld tokens of N=%lld heads are too many", (long long)p->T, (long long)p->N);
    return MSDA_OK;
}

// ---- attention ----

msda_status check_attention(msda_dtype dt, int format, const msda_cache_problem* p) {
    msda_status s = check(dt, format, p);
    if (s != MSDA_OK) return s;
    if (p->M < 1 || p->M % p->N) return failf(MSDA_ERR_INVALID_ARG, "N=%lld key heads do not divide M=%lld query heads", (long long)p->N, (long long)p->M);
    if (p->M > 65535) return failf(MSDA_ERR_UNSUPPORTED, "M=%lld too large", (long long)p->M);
    const int64_t G = p->M / p->N;
    // the line of all tiles (16 rows, 64 keys at least) is counted in 32 bits
    const int64_t tiles = (longest_of(p) + 63) / 64 + (p->source + 63) / 64 + 1, rows = (p->T * G + 15) / 16;
    int64_t all;
    if (p->T * G > kMost || !msda::mul_fits(p->B * p->N, rows, &all) || !msda::mul_fits(all, tiles, &all) || all > 0x7fffffffll / 2)
        return failf(MSDA_ERR_UNSUPPORTED, "B=%lld sequences of T=%lld tokens and M=%lld heads over %lld tokens are too many for one call", (long long)p->B,
                     (long long)p->T, (long long)p->M, (long long)p->longest);
    return MSDA_OK;
}

// How a call runs; of its sizes alone.
struct CachePlan {
    msda::CacheRowsShape shape;
    int64_t rows, row_tiles, units, most_tiles;  // most_tiles: of a unit
    int nq;                                      // row tiles of 128 a block on the tensor cores (tcgen05); 0: the kernel of few rows
    int blocks, least, whole;
    size_t part_l2, units_at, bytes;             // workspace: rows, their statistics, where each unit's parts are
};

// Whether TMA can read a tensor's three dimensions at these strides (elements of `es` bytes): whole vectors, checked already, and
// neither broadcast nor 2^40 bytes apart.
bool tma_strides(const int64_t* st, int64_t a, int64_t b, int64_t c, int64_t es) {
    const int64_t n[3] = {a, b, c};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (st[i] == 0 || st[i] * es >= 1ll << 40)) return false;
    return true;
}

// The tensor-core kernel's row tiles: 16-bit queries with more rows a key head than the mma.sync kernel has in a tile (32 rows there
// take two: 8 x 16384 tokens, 4 key heads of 128: bf16 95 us against 61 here, e4m3 75 against 67; 16 rows 61 and 52).  Two row tiles a
// block where one does not hold the rows, unquantised: keys are then read and multiplied for both.  With codes two row tiles leave too
// few registers to convert a tile in its time (256 rows of 64 channels over 16384 tokens: 137 us against 126 as two units).
int tc_tiles(msda_dtype dt, int format, const msda_cache_problem* p, int64_t rows) {
    const int64_t G = p->M / p->N, es = format == MSDA_CACHE_SAME ? 2 : 1;
    if (dt == MSDA_F32 || rows <= 16 || G > msda::kTcRows) return 0;
    if (!tma_strides(p->query_stride, p->B, p->T, p->M, 2 * G)) return 0;
    if (longest_of(p) > 0 && (!tma_strides(p->cache_key_stride, p->pages, p->page, p->N, es) ||
                              !tma_strides(p->cache_value_stride, p->pages, p->page, p->N, es)))
        return 0;
    if (format == MSDA_CACHE_SAME && p->source > 0 &&
        (!tma_strides(p->key_stride, p->B, p->source, p->N, 2) || !tma_strides(p->value_stride, p->B, p->source, p->N, 2)))
        return 0;
    return format == MSDA_CACHE_SAME && rows > msda::kTcRows / G * G ? 2 : 1;
}

CachePlan plan_of(msda_dtype dt, int format, const msda_cache_problem* p) {
    CachePlan c{};
    const int64_t G = p->M / p->N;
    c.rows = p->T * G;
    c.nq = tc_tiles(dt, format, p, c.rows);
    if (c.nq) c.shape = {(int)(c.nq * (msda::kTcRows / G * G)), msda::kTcRows, msda::kTcRows, 1};
    else c.shape = dt == MSDA_F32   ? msda::cache_rows_shape<float>(format, (int)p->D, (int)c.rows)
              : dt == MSDA_F16 ? msda::cache_rows_shape<__half>(format, (int)p->D, (int)c.rows)
                               : msda::cache_rows_shape<__nv_bfloat16>(format, (int)p->D, (int)c.rows);
    c.row_tiles = (c.rows + c.shape.tile_rows - 1) / c.shape.tile_rows;
    c.units = p->B * p->N * c.row_tiles;
    c.most_tiles = (longest_of(p) + c.shape.tile_keys - 1) / c.shape.tile_keys + (p->source + c.shape.tail_keys - 1) / c.shape.tail_keys;
    if (c.most_tiles < 1) c.most_tiles = 1;
    // A block takes `least` tiles at least, and units of up to twice that run whole: a second launch and the parts cost about 6 us (2 x 256
    // tokens 7.5 whole, 13.1 with blocks of 4 tiles).  One token of 16 heads on 4 of 128 channels, bf16, with `least` at half, this, twice,
    // us: 2 x 512 tokens 12.1, 13.0, 15.9, 2 x 4096 15.6, 14.8, 16.4; trees of 16 over 2 x 512 12.7, 15.4, 17.2, over 8 x 4096 25.8
    // each; a binary32 tree of 25 over 8 x 900 22.7, 24.3, 26.5.  Whole up to four times `least`: 2 x 512 10.2, but that tree 31.5.
    c.least = c.nq ? 2 : 4;
    c.whole = c.most_tiles <= 2 * c.least;
    const int64_t most = msda::kPlanSms * c.shape.resident, want = (c.units * c.most_tiles + c.least - 1) / c.least;
    c.blocks = (int)(c.whole ? c.units : want < most ? want : most);
    c.part_l2 = (size_t)c.blocks * 2 * c.shape.tile_rows * p->D * 4;
    c.units_at = c.part_l2 + (size_t)c.blocks * 2 * c.shape.tile_rows * 4;
    c.bytes = c.whole ? 0 : c.units_at + (size_t)c.units * 8;
    return c;
}

template <int F>
cudaError_t launch_tc_format(const CacheArgs& a, msda_dtype dt, int nq, int grid, cudaStream_t st) {
    return dt == MSDA_BF16 ? msda::launch_cache_tc<true, F>(a, nq, grid, st) : msda::launch_cache_tc<false, F>(a, nq, grid, st);
}
cudaError_t launch_tc(const CacheArgs& a, msda_dtype dt, int format, int nq, int grid, cudaStream_t st) {
    if (format == MSDA_CACHE_SAME) return launch_tc_format<msda::kCacheSame>(a, dt, nq, grid, st);
    if (format == MSDA_CACHE_E4M3) return launch_tc_format<msda::kCacheE4m3>(a, dt, nq, grid, st);
    return launch_tc_format<msda::kCacheInt8>(a, dt, nq, grid, st);
}

}  // namespace

extern "C" {

msda_status msda_cache_write(msda_dtype dt, int format, const msda_cache_problem* p, const void* key, const void* value,
                             const int32_t* table, const int32_t* start, const int32_t* counts, const int32_t* select, void* cache_key,
                             void* cache_value, uint8_t* key_scale, uint8_t* value_scale, msda_stream_t stream) {
    msda::clear_error();
    msda_status s = check(dt, format, p);
    if (s != MSDA_OK || (s = move_size(p)) != MSDA_OK) return s;
    if (!select && p->T > p->source)
        return failf(MSDA_ERR_INVALID_ARG, "T=%lld rows of source=%lld tokens without select", (long long)p->T, (long long)p->source);
    const bool rows = p->B > 0 && p->T > 0;
    const size_t es = dt == MSDA_F32 ? 4 : 2;
    if ((s = vectors(key, p->key_stride, p->B, p->source, p->N, es, rows && p->source > 0, "key")) ||
        (s = vectors(value, p->value_stride, p->B, p->source, p->N, es, rows && p->source > 0, "value")) ||
        (s = msda::need_ptr(start, rows, 4, "start")) || (s = msda::need_ptr(counts, counts != nullptr, 4, "counts")) ||
        (s = msda::need_ptr(select, select != nullptr, 4, "select")) ||
        (s = cache_ok(dt, format, p, cache_key, cache_value, key_scale, value_scale, table, rows && p->pages > 0 && p->width > 0)))
        return s;
    if (!rows) return MSDA_OK;
    CacheMoveArgs a{};
    a.c = pages_of(p, cache_key, cache_value, key_scale, value_scale, table);
    a.key = key, a.value = value;
    three(p->key_stride, a.k_sb, a.k_st, a.k_sh);
    three(p->value_stride, a.v_sb, a.v_st, a.v_sh);
    a.first = start, a.counts = counts, a.select = select, a.select_sb = p->select_stride;
    a.B = (int)p->B, a.T = (int)p->T, a.N = (int)p->N, a.D = (int)p->D, a.source = (int)p->source;
    return move(dt, format, a, true, reinterpret_cast<cudaStream_t>(stream));
}

msda_status msda_cache_read(msda_dtype dt, int format, const msda_cache_problem* p, const void* cache_key, const void* cache_value,
                            const uint8_t* key_scale, const uint8_t* value_scale, const int32_t* table, const int32_t* lengths, void* key,
                            void* value, msda_stream_t stream) {
    msda::clear_error();
    msda_status s = check(dt, format, p);
    if (s != MSDA_OK || (s = move_size(p)) != MSDA_OK) return s;
    const bool rows = p->B > 0 && p->T > 0;
    if ((s = msda::need_ptr(key, rows, 16, "key")) || (s = msda::need_ptr(value, rows, 16, "value")) ||
        (s = msda::need_ptr(lengths, rows, 4, "lengths")) ||
        (s = cache_ok(dt, format, p, cache_key, cache_value, key_scale, value_scale, table, rows && p->pages > 0 && p->width > 0)))
        return s;
    if (!rows) return MSDA_OK;
    CacheMoveArgs a{};
    a.c = pages_of(p, cache_key, cache_value, key_scale, value_scale, table);
    a.key = key, a.value = value, a.first = lengths;
    a.B = (int)p->B, a.T = (int)p->T, a.N = (int)p->N, a.D = (int)p->D;
    return move(dt, format, a, false, reinterpret_cast<cudaStream_t>(stream));
}

size_t msda_cache_attention_workspace_size(msda_dtype dt, int format, const msda_cache_problem* p) {
    if (check_attention(dt, format, p) != MSDA_OK || p->B == 0 || p->T == 0) return 0;
    return plan_of(dt, format, p).bytes;
}

msda_status msda_cache_attention(msda_dtype dt, int format, const msda_cache_problem* p, double scale, const void* query,
                                 const void* cache_key, const void* cache_value, const uint8_t* key_scale, const uint8_t* value_scale,
                                 const int32_t* table, const int32_t* lengths, const void* key, const void* value, const uint8_t* mask,
                                 const int32_t* counts, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                 msda_stream_t stream) {
    msda::clear_error();
    msda_status s = check_attention(dt, format, p);
    if (s != MSDA_OK) return s;
    if (!(scale > 0.0 && scale < 1e30)) return failf(MSDA_ERR_INVALID_ARG, "scale=%g must be positive", scale);
    const bool rows = p->B > 0 && p->T > 0, fresh = rows && p->source > 0;
    if (p->source != 0 && p->source != p->T)
        return failf(MSDA_ERR_INVALID_ARG, "source=%lld must be 0 (no new keys) or T=%lld", (long long)p->source, (long long)p->T);
    if (mask && p->source == 0) return failf(MSDA_ERR_INVALID_ARG, "mask is of new tokens, and there are none");
    const size_t es = dt == MSDA_F32 ? 4 : 2;
    if ((s = vectors(query, p->query_stride, p->B, p->T, p->M, es, rows, "query")) ||
        (s = vectors(key, p->key_stride, p->B, p->source, p->N, es, fresh, "key")) ||
        (s = vectors(value, p->value_stride, p->B, p->source, p->N, es, fresh, "value")) || (s = msda::need_ptr(lengths, rows, 4, "lengths")) ||
        (s = msda::need_ptr(counts, counts != nullptr, 4, "counts")) || (s = msda::need_ptr(out, rows, 16, "out")) ||
        (s = msda::need_ptr(lse, rows, 4, "lse")) ||
        (s = cache_ok(dt, format, p, cache_key, cache_value, key_scale, value_scale, table, rows && longest_of(p) > 0)))
        return s;
    if (!rows) return MSDA_OK;
    const CachePlan plan = plan_of(dt, format, p);
    if (plan.bytes && (!workspace || workspace_bytes < plan.bytes || !msda::aligned_to(workspace, 256)))
        return failf(MSDA_ERR_WORKSPACE, "workspace of %zu bytes, 256-byte aligned, needed (got %zu)", plan.bytes, workspace_bytes);
    CacheArgs a{};
    a.c = pages_of(p, cache_key, cache_value, key_scale, value_scale, table);
    if ((s = msda::error_word(&a.c.err)) != MSDA_OK) return s;
    a.lengths = lengths, a.counts = counts;
    a.q = query, a.nk = fresh ? key : nullptr, a.nv = fresh ? value : nullptr, a.mask = mask;
    three(p->query_stride, a.q_sb, a.q_st, a.q_sh);
    three(p->key_stride, a.nk_sb, a.nk_st, a.nk_sh);
    three(p->value_stride, a.nv_sb, a.nv_st, a.nv_sh);
    a.mk_sb = p->mask_stride[0], a.mk_sq = p->mask_stride[1];
    a.B = (int)p->B, a.T = (int)p->T, a.M = (int)p->M, a.N = (int)p->N, a.D = (int)p->D, a.G = (int)(p->M / p->N);
    a.rows = (int)plan.rows, a.row_tiles = (int)plan.row_tiles, a.tile_rows = plan.shape.tile_rows;
    while ((1 << a.tile_log2) < plan.shape.tile_keys) ++a.tile_log2;
    while ((1 << a.tail_log2) < plan.shape.tail_keys) ++a.tail_log2;
    // never 0, by which the -inf of a hidden token would become NaN (a score is then off by 2^-149 |q k|, below 2^-20)
    a.c2 = std::fmax((float)(scale * (double)msda::kLog2e), std::numeric_limits<float>::denorm_min());
    a.out = out, a.lse = lse;
    a.part_o = static_cast<float*>(workspace);  // null where no unit is shared
    a.part_l2 = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + plan.part_l2);
    a.units = reinterpret_cast<int2*>(static_cast<unsigned char*>(workspace) + plan.units_at);
    a.blocks = plan.blocks, a.least = plan.least, a.whole = plan.whole;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    bool traced;
    {
        msda::TraceSpan ts(st);
        traced = ts.slot >= 0;
        const cudaError_t e = plan.nq          ? launch_tc(a, dt, format, plan.nq, plan.blocks, st)
                              : dt == MSDA_F32 ? msda::launch_cache_rows<float>(a, format, plan.blocks, st)
                              : dt == MSDA_F16 ? msda::launch_cache_rows<__half>(a, format, plan.blocks, st)
                                               : msda::launch_cache_rows<__nv_bfloat16>(a, format, plan.blocks, st);
        ts.end(MSDA_KERNEL_CACHE_ATTENTION, p->B * p->M * p->T);
        if ((s = launched(e, "cache attention kernel launch")) != MSDA_OK) return s;
    }
    if (plan.whole) return MSDA_OK;
    msda::TraceSpan ts(st);
    s = launched(msda::launch_cache_join(a, dt, !traced, st), "cache attention join kernel launch");
    ts.end(MSDA_KERNEL_CACHE_JOIN, p->B * p->M * p->T);
    return s;
}

}  // extern "C"
