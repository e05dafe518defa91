// msda_cache.cu -- the paged cache of keys and values: checks and launches of
// msda_cache_write / _read / _attention, the kernels that write and read rows,
// and the one that joins the parts of units which several blocks shared.
//
// Writing and reading are bound by memory: a row of D channels lies in the lanes
// that 16 bytes of the unquantised type each make, so its largest magnitude takes
// log2(lanes) exchanges and every access is a whole vector.  A block takes 16
// tokens of all heads, tokens of a head next to each other in its lanes: the
// cache's side (head by head) is then read or written in runs of 16 rows, the
// other side in whole tokens.
#include <cuda_runtime.h>

#include <cstdint>

#include "msda_cache.cuh"
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
    int lanes, block_log2;  // lanes a row (a power of two); tokens a block of rows (a power of two up to 16)
};

// Row x of a sequence's rows in blocks of 2^k tokens: token fastest, then head, then block.
__device__ __forceinline__ bool cache_row(const CacheMoveArgs& a, unsigned x, int* t, int* n) {
    const unsigned in = x & ((1u << a.block_log2) - 1u), y = x >> a.block_log2, z = y / (unsigned)a.N;
    *n = (int)(y - z * (unsigned)a.N);
    const long long tok = ((long long)z << a.block_log2) + in;
    *t = (int)tok;
    return tok < a.T;
}

template <typename T, int F>
__global__ void __launch_bounds__(kMoveThreads) msda_cache_write_kernel(const CacheMoveArgs a) {
    constexpr int E = CacheVec<T>::n, U = 2;
    const int at = threadIdx.x & (a.lanes - 1), rows = kMoveThreads / a.lanes;
    const bool in = at * E < a.D;
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        const int start = a.first[b], count = cache_count(a.c, a.counts, b, a.T);
        uint4 x[U][2];
        long long to[U][2];
        long long scale[U][2];
        bool on[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            int t, n;
            on[i] = cache_row(a, (blockIdx.x * U + i) * rows + threadIdx.x / a.lanes, &t, &n) && t < count;
            x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
            if (!on[i]) continue;
            const long long token = (long long)start + t;
            int page = -1, src = t;
            if (token >= 0 && token < a.c.longest) page = cache_page(a.c, b, (int)token);
            else atomicOr(a.c.err, kCacheBad);
            if (a.select) {
                src = a.select[b * a.select_sb + t];
                if ((unsigned)src >= (unsigned)a.source) {
                    atomicOr(a.c.err, kCacheBad);
                    page = -1;
                }
            }
            on[i] = page >= 0;
            if (!on[i]) continue;
            const int place = (int)token & (a.c.page - 1);
            if (in) {
                x[i][0] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.key) + b * a.k_sb + src * a.k_st + n * a.k_sh + at * E);
                x[i][1] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.value) + b * a.v_sb + src * a.v_st + n * a.v_sh + at * E);
            }
            to[i][0] = page * a.c.k_sp + place * a.c.k_st + n * a.c.k_sh + at * E;
            to[i][1] = page * a.c.v_sp + place * a.c.v_st + n * a.c.v_sh + at * E;
            scale[i][0] = page * a.c.ks_sp + place * a.c.ks_st + n * a.c.ks_sh;
            scale[i][1] = page * a.c.vs_sp + place * a.c.vs_st + n * a.c.vs_sh;
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                void* base = w ? a.c.v : a.c.k;
                if constexpr (F == kCacheSame) {
                    if (on[i] && in) *reinterpret_cast<uint4*>(static_cast<T*>(base) + to[i][w]) = x[i][w];
                } else {
                    float v[E];
                    CacheVec<T>::get(x[i][w], v);
                    uint32_t top = 0;  // of non-negative floats the bits are in order, and NaN is above infinity
#pragma unroll
                    for (int e = 0; e < E; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
                    for (int s = a.lanes >> 1; s > 0; s >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, s));
                    const uint32_t byte = cache_scale_byte<F>(__uint_as_float(top));
                    const float up = byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
                    uint32_t codes[E / 4];
#pragma unroll
                    for (int e = 0; e < E / 4; ++e) {
                        codes[e] = byte == 255u ? 0u : cache_codes<F>(v[4 * e] * up, v[4 * e + 1] * up, v[4 * e + 2] * up, v[4 * e + 3] * up);
                    }
                    if (on[i]) {
                        uint8_t* p = static_cast<uint8_t*>(base) + to[i][w];
                        if (in) {
                            if constexpr (E == 8) *reinterpret_cast<uint2*>(p) = make_uint2(codes[0], codes[1]);
                            else *reinterpret_cast<uint32_t*>(p) = codes[0];
                        }
                        if (at == 0) (w ? a.c.vs : a.c.ks)[scale[i][w]] = (uint8_t)byte;
                    }
                }
            }
    }
}

template <typename T, int F>
__global__ void __launch_bounds__(kMoveThreads) msda_cache_read_kernel(const CacheMoveArgs a) {
    constexpr int E = CacheVec<T>::n, U = 4;
    const int at = threadIdx.x & (a.lanes - 1), rows = kMoveThreads / a.lanes;
    const bool in = at * E < a.D;
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        const int length = cache_length(a.c, a.first, b);
        uint4 x[U][2];
        uint32_t scale[U][2];
        long long to[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            int t, n;
            const bool row = cache_row(a, (blockIdx.x * U + i) * rows + threadIdx.x / a.lanes, &t, &n);
            x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
            scale[i][0] = scale[i][1] = 0;
            to[i] = row && in ? (((long long)b * a.T + t) * a.N + n) * a.D + at * E : -1;
            if (!row || t >= length) continue;
            const int page = cache_page(a.c, b, t);
            if (page < 0) continue;
            const int place = t & (a.c.page - 1);
            const long long k = page * a.c.k_sp + place * a.c.k_st + n * a.c.k_sh + at * E;
            const long long v = page * a.c.v_sp + place * a.c.v_st + n * a.c.v_sh + at * E;
            if constexpr (F == kCacheSame) {
                if (in) {
                    x[i][0] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.c.k) + k);
                    x[i][1] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.c.v) + v);
                }
            } else {
                if (in) {
                    const uint8_t *kp = static_cast<const uint8_t*>(a.c.k) + k, *vp = static_cast<const uint8_t*>(a.c.v) + v;
                    if constexpr (E == 8) {
                        const uint2 p = *reinterpret_cast<const uint2*>(kp), q = *reinterpret_cast<const uint2*>(vp);
                        x[i][0].x = p.x, x[i][0].y = p.y, x[i][1].x = q.x, x[i][1].y = q.y;
                    } else {
                        x[i][0].x = *reinterpret_cast<const uint32_t*>(kp), x[i][1].x = *reinterpret_cast<const uint32_t*>(vp);
                    }
                }
                scale[i][0] = a.c.ks[page * a.c.ks_sp + place * a.c.ks_st + n * a.c.ks_sh];
                scale[i][1] = a.c.vs[page * a.c.vs_sp + place * a.c.vs_st + n * a.c.vs_sh];
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (to[i] < 0) continue;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                T* out = static_cast<T*>(const_cast<void*>(w ? a.value : a.key)) + to[i];
                if constexpr (F == kCacheSame) {
                    *reinterpret_cast<uint4*>(out) = x[i][w];
                } else {
                    const uint32_t c[2] = {x[i][w].x, x[i][w].y};
                    const bool none = scale[i][w] == 255u;
                    const float s = cache_scale(scale[i][w]);
                    float v[E];
#pragma unroll
                    for (int e = 0; e < E / 4; ++e) {
                        uint32_t lo, hi;
                        cache_four_f16<F>(c[e], lo, hi);
                        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&lo)), q = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                        v[4 * e] = p.x * s, v[4 * e + 1] = p.y * s, v[4 * e + 2] = q.x * s, v[4 * e + 3] = q.y * s;
                    }
                    // a code may be rounded up past the type's range: finite rows stay finite
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        v[e] = none ? __uint_as_float(0x7fffffffu) : fminf(fmaxf(v[e], -CacheVec<T>::most()), CacheVec<T>::most());
                    *reinterpret_cast<uint4*>(out) = CacheVec<T>::put(v);
                }
            }
        }
    }
}

// A block a unit (and 32 rows of it): the parts of the blocks that shared it, in their order.  A row's parts lie a slot apart; a
// warp takes a row, a lane its channels.
template <typename T>
__global__ void __launch_bounds__(128) msda_cache_join_kernel(const CacheArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long id = blockIdx.x;
    const int rt = (int)(id % a.row_tiles);
    id /= a.row_tiles;
    const int n = (int)(id % a.N), b = (int)(id / a.N);
    long long x;
    const long long share = cache_share(a, cache_all_tiles(a, b, &x));
    CacheUnit u;
    cache_unit_at(a, b, n, 0, u);
    if (n > 0) x += cache_head_tiles(a, b) * n;
    for (; u.rt < rt; ++u.rt, cache_unit_tiles(a, u)) x += u.tiles;
    const long long c0 = x / share, c1 = (x + u.tiles - 1) / share;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // launched as a programmatic dependent of the kernel that makes the parts
    if (c0 == c1) return;
    for (int r = blockIdx.y * 32 + warp; r < min(a.tile_rows, (int)(blockIdx.y + 1) * 32); r += 4) {
        const int row = rt * a.tile_rows + r, t = row / a.G;
        if (row >= a.rows) return;
        auto slot = [&](long long c) { return (2 * c + (c == c0 && x != c0 * share ? 1 : 0)) * a.tile_rows + r; };
        float top = -attn_inf();
        bool nan = false;
        for (long long c = c0 + lane; c <= c1; c += 32) {
            const float l2 = a.part_l2[slot(c)];
            top = fmaxf(top, l2), nan |= l2 != l2;
        }
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        if (__any_sync(0xffffffffu, nan)) top = __uint_as_float(0x7fffffffu);
        float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
        for (long long c = c0; c <= c1; ++c) {
            const long long at = slot(c);
            const float w = top == -attn_inf() ? 0.f : exp2f(a.part_l2[at] - top);
            sum += w;
            if (lane * 4 < a.D) {
                const float4 y = *reinterpret_cast<const float4*>(a.part_o + at * a.D + lane * 4);
                o[0] += w * y.x, o[1] += w * y.y, o[2] += w * y.z, o[3] += w * y.w;
            }
        }
        const int h = n * a.G + row - t * a.G;
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
        if (lane == 0) a.lse[((long long)b * a.M + h) * a.T + t] = sum == 0.f ? -attn_inf() : (top + log2f(sum)) * kLn2;
    }
}

template <typename T>
static cudaError_t join_go(const CacheArgs& a, bool early, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.B * a.N * a.row_tiles), (unsigned)((a.tile_rows + 31) / 32));
    cfg.blockDim = dim3(128);
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
    c.pages = (int)p->pages, c.page = (int)p->page, c.longest = (int)p->longest;
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
    a.lanes = 2;
    while (a.lanes * vec < a.D) a.lanes *= 2;
    a.block_log2 = 0;
    while (a.block_log2 < 4 && (1 << a.block_log2) < a.T) ++a.block_log2;
    const long long blocks = ((long long)a.T + (1 << a.block_log2) - 1) >> a.block_log2, rows = (blocks * a.N) << a.block_log2;
    const long long each = (long long)(msda::kMoveThreads / a.lanes) * (write ? 2 : 4);
    const dim3 grid((unsigned)((rows + each - 1) / each), (unsigned)(a.B < 65535 ? a.B : 65535));
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
    if (p->T * G > kMost || p->B * p->N * ((p->T * G + 15) / 16) > 0x7fffffffll / 2)
        return failf(MSDA_ERR_UNSUPPORTED, "B=%lld sequences of T=%lld tokens and M=%lld heads are too many", (long long)p->B, (long long)p->T, (long long)p->M);
    return MSDA_OK;
}

// How a call runs; of its sizes alone.
struct CachePlan {
    msda::CacheRowsShape shape;
    int64_t rows, row_tiles, units, most_tiles;  // most_tiles: of a unit
    int blocks, least, whole;
    size_t bytes;
};
CachePlan plan_of(msda_dtype dt, int format, const msda_cache_problem* p) {
    CachePlan c{};
    c.rows = p->T * (p->M / p->N);
    c.shape = dt == MSDA_F32   ? msda::cache_rows_shape<float>(format, (int)p->D, (int)c.rows)
              : dt == MSDA_F16 ? msda::cache_rows_shape<__half>(format, (int)p->D, (int)c.rows)
                               : msda::cache_rows_shape<__nv_bfloat16>(format, (int)p->D, (int)c.rows);
    c.row_tiles = (c.rows + c.shape.tile_rows - 1) / c.shape.tile_rows;
    c.units = p->B * p->N * c.row_tiles;
    c.most_tiles = (p->longest + c.shape.tile_keys - 1) / c.shape.tile_keys + (p->source + c.shape.tail_keys - 1) / c.shape.tail_keys;
    if (c.most_tiles < 1) c.most_tiles = 1;
    c.least = 4;
    c.whole = c.most_tiles <= 2 * c.least;
    const int64_t most = msda::kPlanSms * c.shape.resident, want = (c.units * c.most_tiles + c.least - 1) / c.least;
    c.blocks = (int)(c.whole ? c.units : want < most ? want : most);
    c.bytes = c.whole ? 0 : (size_t)c.blocks * 2 * c.shape.tile_rows * (p->D + 1) * 4;
    return c;
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
        (s = cache_ok(dt, format, p, cache_key, cache_value, key_scale, value_scale, table, rows && p->pages > 0 && p->longest > 0)))
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
    a.tile_keys = plan.shape.tile_keys, a.tail_keys = plan.shape.tail_keys;
    a.c2 = (float)(scale * (double)msda::kLog2e);
    a.out = out, a.lse = lse;
    a.part_o = static_cast<float*>(workspace);
    a.part_l2 = a.part_o + (size_t)plan.blocks * 2 * plan.shape.tile_rows * p->D;
    a.blocks = plan.blocks, a.least = plan.least, a.whole = plan.whole;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    bool traced;
    {
        msda::TraceSpan ts(st);
        traced = ts.slot >= 0;
        const cudaError_t e = dt == MSDA_F32   ? msda::launch_cache_rows<float>(a, format, plan.blocks, st)
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
