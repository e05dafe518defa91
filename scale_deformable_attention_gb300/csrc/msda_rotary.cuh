// msda_rotary.cuh -- rotary positions with several axes, and the norm of
// queries and keys per head with that rotation in the same pass.
//
// Rotation: pair j of a head's channels turns by the angle t_j = p[axis(j)] * f[j]:
//   (u, v) -> (u cos t - v sin t, v cos t + u sin t),
// its channels being (j, j + P) or, interleaved, (2j, 2j + 1); channels from 2P
// on pass through.  Norm: r = (mean x^2 + eps)^-1/2, z = x r w, y = R z.
// Gradients, with dz = R^T dy (the rotation by -t) and n = x r:
//   dx = r (w dz - n mean(n w dz)),   dw = sum over rows of n dz.
//
// What bounds it: memory, then issue.  Every element is read once (twice in the
// backward: x and dy) and written once, at 55 % of the DRAM's rate under a
// profiler with 63 to 71 % of the issue slots taken (conversions and selects on
// the ALU 39 to 45 %, FMA pipe 26 to 31 %) by 16 to 28 warps an SM.  All heads of a token share its angles, so in the
// vector form a lane owns 16 bytes of channels of one token, works out their cos
// and sin once in registers and walks the heads: several 16-byte loads in
// flight a lane, no shared memory, no barrier.  In halves a pair's two channels
// belong to two lanes: each works out half of the pair's angles, and the raw 16
// bytes are exchanged by four shuffles a row.  A row's sums take log2(lanes)
// shuffles.  (With the angles of a chunk of tokens in shared memory and a lane
// holding both halves of its pairs, a call of 20 heads of 128 ran at 26 % of the
// copy rate.)  The weights' gradients stay in registers over all rows of a lane,
// then go through one partial row a block and a second kernel that adds the
// partials in a fixed order: no atomics.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace msda {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryMaxAxes = 4;
constexpr int kRotaryMaxChannels = 256;

struct RotaryTensor {
    const void* x;     // input rows (strided)
    const void* dy;    // backward: gradient of the output rows (dense); null forward
    void* y;           // output rows (dense)
    const void* w;     // weight [D], null without norm
    long long sb, ss, sh;  // strides of x in elements: batch, token, head
    int heads;
};

struct RotaryArgs {
    RotaryTensor t[2];  // queries, keys (heads = 0: absent)
    const void* pos;    // [Bp, S, A]
    const float* freq;  // [P]
    float* partial;     // backward: [grid][2][D]
    long long pos_sb;   // batch stride of pos in elements (0: shared)
    int pos_type;       // 0 float32, 1 int32, 2 int64
    int S, D, P, A;
    int axis_end[kRotaryMaxAxes];  // pairs below axis_end[a] (and not below axis_end[a-1]) turn by axis a
    int T;              // element form: tokens a chunk, chunks
    int chunks_per_b;
    long long chunks;
    long long tokens;   // vector form: B * S, and the heads in `parts` parts of `per` (a warp takes one)
    int parts, per;
    float eps, inv_d, sign;
};

template <typename T>
struct Vec16;  // 16 bytes of T
template <>
struct Vec16<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const float* p, float* v) {
        const float4 a = *reinterpret_cast<const float4*>(p);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    }
    static __device__ __forceinline__ void store(float* p, const float* v) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <>
struct Vec16<__half> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const __half* p, float* v) {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ void store(__half* p, const float* v) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <>
struct Vec16<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* v) {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};

template <typename T>
__device__ __forceinline__ float to_f32(T v) { return (float)v; }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// (p + rest) * f near [-pi, pi]: the product as two binary64 numbers, 2 pi as
// two; good for products below 2^51 (n and the difference are held exactly).
// Not inlined: few positions need it, and beside the other path's it cost the
// rotation alone 3 %.
static __device__ __noinline__ float far_angle(double p, double rest, float f) {
    const double t = p * (double)f, lo = fma(p, (double)f, -t) + rest * (double)f;
    const double n = rint(t * 0.15915494309189535);
    double d = fma(-n, 6.283185307179586, t);
    d = fma(-n, 2.4492935982947064e-16, d);
    return (float)(d + lo);
}

// p * f for |p * f| < 2^23, near [-pi, pi].  The product of two binary32 numbers
// is held exactly as hi + lo; n times 2 pi is subtracted, taken as two binary32
// parts (Cody and Waite's reduction): the first subtraction is exact (both sides
// are multiples of the smaller one's last place and the difference is below 4),
// what 2 pi has behind its second part is below 2^-27 after n, so the angle is
// off by its own rounding to binary32 alone.
__device__ __forceinline__ float near_angle(float hi, float p, float f) {
    const float lo = fmaf(p, f, -hi);
    const float n = rintf(hi * 0.15915494309189535f);
    float r = fmaf(-n, 6.2831854820251465f, hi);  // binary32 nearest to 2 pi
    r = fmaf(-n, -1.7484555314695172e-07f, r);    // the rest of 2 pi
    return r + lo;
}

enum { ROT_SCALAR = 0, ROT_HALVES = 1, ROT_INTERLEAVED = 2 };

// cos and sin of pair j of the token whose positions start at element `at`
__device__ __forceinline__ void rotary_angle(const RotaryArgs& a, long long at, int j, float* c, float* s) {
    int ax = 0;
    while (ax < a.A - 1 && j >= a.axis_end[ax]) ++ax;
    const float f = a.freq[j];
    float r;
    if (a.pos_type == 0) {
        const float p = static_cast<const float*>(a.pos)[at + ax], hi = p * f;
        r = fabsf(hi) < 8388608.f ? near_angle(hi, p, f) : far_angle(p, 0.0, f);
    } else {
        const long long v = a.pos_type == 1 ? (long long)static_cast<const int*>(a.pos)[at + ax]
                                            : static_cast<const long long*>(a.pos)[at + ax];
        const float p = (float)v, hi = p * f;
        if (v > -16777217ll && v < 16777217ll && fabsf(hi) < 8388608.f) {
            r = near_angle(hi, p, f);
        } else {  // what binary64 leaves of the position: its upper half is a multiple of 2^32, near p64
            const double p64 = (double)v;
            r = far_angle(p64, fma((double)(v >> 32), 4294967296.0, -p64) + (double)(v & 0xffffffffll), f);
        }
    }
    sincosf(r, s, c);
    *s *= a.sign;
}

// A lane's channels [c, c + V) of a token and what turns them: channel i becomes
//   own_i * cs[i] + other_i * sn[i]
// with `other` the channel it is paired with (interleaved: its neighbour).
template <int V>
struct RotaryLane {
    int c, src;   // first channel; the lane that holds the other halves (halves)
    bool on;      // channels inside D
    float cs[V], sn[V];
};

template <int MODE, int V>
__device__ __forceinline__ void rotary_lane(const RotaryArgs& a, int lg, long long token, RotaryLane<V>& r) {
    const int lane = threadIdx.x & 31, l = lane & ((1 << lg) - 1);
    r.c = l * V;
    r.on = r.c < a.D && token < a.tokens;
    r.src = lane;
#pragma unroll
    for (int i = 0; i < V; ++i) r.cs[i] = 1.f, r.sn[i] = 0.f;
    long long at = 0;
    if (token < a.tokens) {
        const long long b = token / a.S;
        at = b * a.pos_sb + (token - b * a.S) * a.A;
    }
    if constexpr (MODE == ROT_INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const int j = (r.c + i) >> 1;
            if (r.on && j < a.P) {
                float c, s;
                rotary_angle(a, at, j, &c, &s);
                r.cs[i] = r.cs[i + 1] = c;
                r.sn[i] = -s, r.sn[i + 1] = s;
            }
        }
    } else {
        const bool first = r.c < a.P, second = !first && r.c < 2 * a.P;
        if (first) r.src = lane + a.P / V;
        if (second) r.src = lane - a.P / V;
        const int j0 = first ? r.c : r.c - a.P;
        float c[V / 2], s[V / 2];  // the first half's lane takes pairs j0 .. j0 + V/2, the second's the rest
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            c[i] = 1.f, s[i] = 0.f;
            if (r.on && (first || second)) rotary_angle(a, at, j0 + (first ? 0 : V / 2) + i, &c[i], &s[i]);
        }
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float oc = __shfl_sync(0xffffffffu, c[i], r.src), os = __shfl_sync(0xffffffffu, s[i], r.src);
            if (first || second) {
                r.cs[i] = first ? c[i] : oc;
                r.cs[V / 2 + i] = first ? oc : c[i];
                const float lo = first ? s[i] : os, hi = first ? os : s[i];
                r.sn[i] = first ? -lo : lo;
                r.sn[V / 2 + i] = first ? -hi : hi;
            }
        }
    }
}

// the paired channels' values (halves: from the other lane, as raw 16 bytes)
template <typename T, int MODE>
__device__ __forceinline__ uint4 rotary_other(uint4 v, int src) {
    if constexpr (MODE == ROT_INTERLEAVED) return v;
    return make_uint4(__shfl_sync(0xffffffffu, v.x, src), __shfl_sync(0xffffffffu, v.y, src),
                      __shfl_sync(0xffffffffu, v.z, src), __shfl_sync(0xffffffffu, v.w, src));
}

template <typename T>
__device__ __forceinline__ void rotary_unpack(uint4 u, float* v) {
    alignas(16) T t[Vec16<T>::N];
    *reinterpret_cast<uint4*>(t) = u;
    Vec16<T>::load(t, v);
}

// Heads [h0, h1) of one tensor for the warp's tokens.
template <typename T, int MODE, bool NORM, bool BWD>
__device__ __forceinline__ void rotary_heads(const RotaryArgs& a, const RotaryTensor& t, int lg, long long token,
                                             const RotaryLane<Vec16<T>::N>& r, int h0, int h1, float* dw) {
    constexpr int V = Vec16<T>::N;
    // rows worked on at once; with the norm as many more are loaded meanwhile (backward of 20
    // heads of 128: 438 us, 504 without the loads ahead, 467 with one row at once)
    constexpr int U = NORM ? 2 : 4;
    if (h0 >= h1) return;           // the same for the whole warp (no keys: their pointers are null)
    const long long b = token / a.S, s = token - b * a.S;
    const T* x = static_cast<const T*>(t.x) + b * t.sb + s * t.ss + r.c;
    T* y = static_cast<T*>(t.y) + token * t.heads * a.D + r.c;
    const T* dy = BWD ? static_cast<const T*>(t.dy) + token * t.heads * a.D + r.c : nullptr;
    // forward: what multiplies the own channels and the paired ones, weights included; backward: the weights
    float w[V], wo[BWD ? 1 : V];
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = 1.f;
    if constexpr (NORM) {
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (r.c < a.D) raw = *reinterpret_cast<const uint4*>(static_cast<const T*>(t.w) + r.c);
        rotary_unpack<T>(raw, w);
        if constexpr (!BWD) {
            float o[V];
            rotary_unpack<T>(rotary_other<T, MODE>(raw, r.src), o);
#pragma unroll
            for (int i = 0; i < V; ++i) wo[i] = o[MODE == ROT_INTERLEAVED ? i ^ 1 : i] * r.sn[i];
        }
    } else if constexpr (!BWD) {
#pragma unroll
        for (int i = 0; i < V; ++i) wo[i] = r.sn[i];
    }
    if constexpr (!BWD) {
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] *= r.cs[i];
    }
    uint4 xn[U], gn[BWD ? U : 1];
    // A row that does not exist (heads end inside a step, tokens inside a warp) holds values near 1 in each type: zeros would,
    // without eps, make its 1 / sqrt(0) times 0 a NaN in the weights' sums.  (Its factor set to 0 instead: 745 us for
    // 737, 8 x 16641 tokens of 20 heads of 128, both directions.)
    const uint32_t none = BWD && r.c < a.D ? 0x3f803f80u : 0u;
    auto fetch = [&](int h) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = r.on && h + u < h1;
            xn[u] = make_uint4(none, none, none, none);
            if (in) xn[u] = *reinterpret_cast<const uint4*>(x + (h + u) * t.sh);
            if constexpr (BWD) {
                gn[u] = make_uint4(0, 0, 0, 0);
                if (in) gn[u] = *reinterpret_cast<const uint4*>(dy + (long long)(h + u) * a.D);
            }
        }
    };
    if constexpr (NORM) fetch(h0);  // the rotation alone: four rows at once (59 us a direction of the clip), 67 with loads ahead
#pragma unroll 1
    for (int h = h0; h < h1; h += U) {
        if constexpr (!NORM) fetch(h);
        uint4 xr[U], gr[BWD ? U : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            xr[u] = xn[u];
            if constexpr (BWD) gr[u] = gn[u];
        }
        if (NORM && h + U < h1) fetch(h + U);
        float rn[U];
        if constexpr (NORM) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float v[V], ss = 0.f;
                rotary_unpack<T>(xr[u], v);
#pragma unroll
                for (int i = 0; i < V; ++i) ss = fmaf(v[i], v[i], ss);
                rn[u] = ss;
            }
            for (int o = (1 << lg) >> 1; o > 0; o >>= 1) {
#pragma unroll
                for (int u = 0; u < U; ++u) rn[u] += __shfl_xor_sync(0xffffffffu, rn[u], o);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) rn[u] = rsqrtf(rn[u] * a.inv_d + a.eps);
        }
        if constexpr (!BWD) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float v[V], o[V], z[V];
                const uint4 other = rotary_other<T, MODE>(xr[u], r.src);
                rotary_unpack<T>(xr[u], v);
                rotary_unpack<T>(other, o);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    z[i] = fmaf(v[i], w[i], o[MODE == ROT_INTERLEAVED ? i ^ 1 : i] * wo[i]);
                    if constexpr (NORM) z[i] *= rn[u];
                }
                if (r.on && h + u < h1) Vec16<T>::store(y + (long long)(h + u) * a.D, z);
            }
        } else {
            float dot[U], g[U][V], n[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float o[V];
                const uint4 other = rotary_other<T, MODE>(gr[u], r.src);
                rotary_unpack<T>(gr[u], g[u]);
                rotary_unpack<T>(other, o);
                rotary_unpack<T>(xr[u], n[u]);
                dot[u] = 0.f;
                float z[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    z[i] = fmaf(g[u][i], r.cs[i], -o[MODE == ROT_INTERLEAVED ? i ^ 1 : i] * r.sn[i]);  // turned back
                    n[u][i] *= rn[u];
                    dw[i] = fmaf(z[i], n[u][i], dw[i]);
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    g[u][i] = z[i] * w[i];
                    dot[u] = fmaf(g[u][i], n[u][i], dot[u]);
                }
            }
            for (int o = (1 << lg) >> 1; o > 0; o >>= 1) {
#pragma unroll
                for (int u = 0; u < U; ++u) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], o);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                dot[u] *= a.inv_d;
#pragma unroll
                for (int i = 0; i < V; ++i) g[u][i] = rn[u] * fmaf(-n[u][i], dot[u], g[u][i]);
                if (r.on && h + u < h1) Vec16<T>::store(y + (long long)(h + u) * a.D, g[u]);
            }
        }
    }
}

// Element form, for rows that 16-byte vectors do not fit: a warp takes a row,
// lane l the pairs l, l + 32, ... and then the channels behind them.
// dw: the lane's sums, [4 pairs][2] and [8 channels behind].
template <typename T, bool NORM, bool BWD>
__device__ __forceinline__ void rotary_rows_scalar(const RotaryArgs& a, const RotaryTensor& t, bool inter, long long b,
                                                   int s0, int nt, const float2* table, float* dw) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T* x = static_cast<const T*>(t.x) + b * t.sb + (long long)s0 * t.ss;
    const long long dense0 = (b * a.S + s0) * (long long)t.heads * a.D;
    T* y = static_cast<T*>(t.y) + dense0;
    const T* dy = BWD ? static_cast<const T*>(t.dy) + dense0 : nullptr;
    const T* w = static_cast<const T*>(t.w);
    const int rows = nt * t.heads;
    for (int row = warp; row < rows; row += kRotaryThreads / 32) {
        const int tok = row / t.heads, head = row - tok * t.heads;
        const T* px = x + (long long)tok * t.ss + (long long)head * t.sh;
        T* py = y + (long long)row * a.D;
        const T* pg = BWD ? dy + (long long)row * a.D : nullptr;
        const float2* tab = table + tok * a.P;
        float r = 1.f, dot = 0.f;
        if constexpr (NORM) {
            float ss = 0.f;
            for (int c = lane; c < a.D; c += 32) {
                const float v = to_f32(px[c]);
                ss = fmaf(v, v, ss);
            }
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            r = rsqrtf(ss * a.inv_d + a.eps);
        }
        float zu[4], zv[4], zp[8];  // D <= 256: at most 4 pairs and 8 channels behind them a lane
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = lane + 32 * i;
            zu[i] = zv[i] = 0.f;
            if (j < a.P) {
                const int cu = inter ? 2 * j : j, cv = inter ? 2 * j + 1 : j + a.P;
                const float2 cs = tab[j];
                if constexpr (!BWD) {
                    const float u = to_f32(px[cu]) * (NORM ? r * to_f32(w[cu]) : 1.f);
                    const float v = to_f32(px[cv]) * (NORM ? r * to_f32(w[cv]) : 1.f);
                    py[cu] = from_f32<T>(u * cs.x - v * cs.y);
                    py[cv] = from_f32<T>(v * cs.x + u * cs.y);
                } else {
                    const float gu = to_f32(pg[cu]), gv = to_f32(pg[cv]);
                    const float du = gu * cs.x + gv * cs.y, dv = gv * cs.x - gu * cs.y;
                    const float nu = to_f32(px[cu]) * r, nv = to_f32(px[cv]) * r;
                    dw[2 * i] = fmaf(du, nu, dw[2 * i]);
                    dw[2 * i + 1] = fmaf(dv, nv, dw[2 * i + 1]);
                    zu[i] = du * to_f32(w[cu]);
                    zv[i] = dv * to_f32(w[cv]);
                    dot = fmaf(zu[i], nu, fmaf(zv[i], nv, dot));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = 2 * a.P + lane + 32 * i;
            zp[i] = 0.f;
            if (c < a.D) {
                if constexpr (!BWD) {
                    py[c] = from_f32<T>(to_f32(px[c]) * (NORM ? r * to_f32(w[c]) : 1.f));
                } else {
                    const float g = to_f32(pg[c]), n = to_f32(px[c]) * r;
                    dw[8 + i] = fmaf(g, n, dw[8 + i]);
                    zp[i] = g * to_f32(w[c]);
                    dot = fmaf(zp[i], n, dot);
                }
            }
        }
        if constexpr (BWD) {
            for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
            dot *= a.inv_d;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = lane + 32 * i;
                if (j < a.P) {
                    const int cu = inter ? 2 * j : j, cv = inter ? 2 * j + 1 : j + a.P;
                    py[cu] = from_f32<T>(r * fmaf(-to_f32(px[cu]) * r, dot, zu[i]));
                    py[cv] = from_f32<T>(r * fmaf(-to_f32(px[cv]) * r, dot, zv[i]));
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = 2 * a.P + lane + 32 * i;
                if (c < a.D) py[c] = from_f32<T>(r * fmaf(-to_f32(px[c]) * r, dot, zp[i]));
            }
        }
    }
}

// Vector form: a warp takes 32 >> lg tokens and one part of the heads (queries'
// heads, then keys'); persistent.  Element form: a block takes chunks of T
// tokens of one batch item, with their cos and sin in shared memory (float2[T][P]).
// Shared memory is reused as float[8][D] for the weights' gradients at the end.
template <typename T, int MODE, bool NORM, bool BWD>
__global__ void __launch_bounds__(kRotaryThreads, MODE == ROT_SCALAR || BWD ? 2 : 3) msda_rotary_kernel(const RotaryArgs a, int lg, bool inter) {
    extern __shared__ __align__(16) unsigned char rotary_smem[];
    constexpr int V = Vec16<T>::N;
    constexpr int W = MODE == ROT_SCALAR ? 16 : V;
    float dw[2][BWD ? W : 1];
    if constexpr (BWD) {
#pragma unroll
        for (int i = 0; i < W; ++i) dw[0][i] = dw[1][i] = 0.f;
    }
    if constexpr (MODE == ROT_SCALAR) {
        float2* table = reinterpret_cast<float2*>(rotary_smem);
        for (long long ch = blockIdx.x; ch < a.chunks; ch += gridDim.x) {
            const long long b = ch / a.chunks_per_b;
            const int s0 = (int)(ch - b * a.chunks_per_b) * a.T;
            const int nt = min(a.T, a.S - s0);
            __syncthreads();  // the table of the chunk before is no longer read
            for (int i = threadIdx.x; i < nt * a.P; i += kRotaryThreads) {
                const int t = i / a.P, j = i - t * a.P;
                rotary_angle(a, b * a.pos_sb + (long long)(s0 + t) * a.A, j, &table[i].x, &table[i].y);
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (a.t[k].heads > 0) rotary_rows_scalar<T, NORM, BWD>(a, a.t[k], inter, b, s0, nt, table, dw[k]);
        }
    } else {
        const int tw = 32 >> lg;
        const long long groups = (a.tokens + tw - 1) / tw, items = groups * a.parts;
        const long long stride = (long long)gridDim.x * (kRotaryThreads / 32);
        for (long long it = (long long)blockIdx.x * (kRotaryThreads / 32) + (threadIdx.x >> 5); it < items; it += stride) {
            const long long group = it / a.parts;
            const int h0 = (int)(it - group * a.parts) * a.per, h1 = h0 + a.per;
            const long long token = group * tw + ((threadIdx.x & 31) >> lg);
            RotaryLane<V> r;
            rotary_lane<MODE, V>(a, lg, token, r);
            const long long safe = token < a.tokens ? token : a.tokens - 1;  // a lane past the end reads and writes nothing
            const int M = a.t[0].heads, all = M + a.t[1].heads;
            rotary_heads<T, MODE, NORM, BWD>(a, a.t[0], lg, safe, r, min(h0, M), min(h1, M), dw[0]);
            rotary_heads<T, MODE, NORM, BWD>(a, a.t[1], lg, safe, r, max(h0, M) - M, max(min(h1, all), M) - M, dw[1]);
        }
    }
    if constexpr (BWD) {
        // the block's sums of both weights' gradients: lanes of a warp that own
        // the same channels, then the warps, each in a fixed order
        float* red = reinterpret_cast<float*>(rotary_smem);  // [warps][D]
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            __syncthreads();
            if constexpr (MODE == ROT_SCALAR) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = lane + 32 * i;
                    if (j < a.P) {
                        red[warp * a.D + (inter ? 2 * j : j)] = dw[k][2 * i];
                        red[warp * a.D + (inter ? 2 * j + 1 : j + a.P)] = dw[k][2 * i + 1];
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int c = 2 * a.P + lane + 32 * i;
                    if (c < a.D) red[warp * a.D + c] = dw[k][8 + i];
                }
            } else {
                const int c = (lane & ((1 << lg) - 1)) * V;
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    float v = dw[k][i];
                    for (int o = 1 << lg; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                    if (lane < (1 << lg) && c < a.D) red[warp * a.D + c + i] = v;
                }
            }
            __syncthreads();
            for (int c = threadIdx.x; c < a.D; c += kRotaryThreads) {
                float v = 0.f;
                for (int q = 0; q < kRotaryThreads / 32; ++q) v += red[q * a.D + c];
                a.partial[((long long)blockIdx.x * 2 + k) * a.D + c] = v;
            }
        }
    }
}

// Weights' gradients: partial[n][2][D] added over n in a fixed order, rounded once.
template <typename T>
__global__ void __launch_bounds__(1024) msda_rotary_weight_kernel(const float* partial, int n, int D, T* dwq, T* dwk) {
    __shared__ float red[32][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
    float v = 0.f;
    if (col < 2 * D)
#pragma unroll 4
        for (int i = part; i < n; i += 32) v += partial[(long long)i * 2 * D + col];
    red[part][threadIdx.x & 31] = v;
    __syncthreads();
    if (part == 0 && col < 2 * D) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x & 31];
        if (col < D) {
            if (dwq) dwq[col] = from_f32<T>(s);
        } else if (dwk) {
            dwk[col - D] = from_f32<T>(s);
        }
    }
}

// One call's kernels for dtype T (each in its own translation unit).
template <typename T>
cudaError_t launch_rotary(const RotaryArgs& a, int mode, bool norm, bool bwd, int lg, bool inter, unsigned grid,
                          size_t smem, cudaStream_t st);
template <typename T>
cudaError_t launch_rotary_weight(const float* partial, int n, int D, void* dwq, void* dwk, cudaStream_t st);

#ifdef MSDA_ROTARY_INSTANTIATE
template <typename T>
cudaError_t launch_rotary(const RotaryArgs& a, int mode, bool norm, bool bwd, int lg, bool inter, unsigned grid,
                          size_t smem, cudaStream_t st) {
#define MSDA_ROTARY_GO(MODE)                                                                                    \
    do {                                                                                                        \
        if (bwd) msda_rotary_kernel<T, MODE, true, true><<<grid, kRotaryThreads, smem, st>>>(a, lg, inter);     \
        else if (norm) msda_rotary_kernel<T, MODE, true, false><<<grid, kRotaryThreads, smem, st>>>(a, lg, inter); \
        else msda_rotary_kernel<T, MODE, false, false><<<grid, kRotaryThreads, smem, st>>>(a, lg, inter);       \
    } while (0)
    switch (mode) {
    case ROT_HALVES: MSDA_ROTARY_GO(ROT_HALVES); break;
    case ROT_INTERLEAVED: MSDA_ROTARY_GO(ROT_INTERLEAVED); break;
    default: MSDA_ROTARY_GO(ROT_SCALAR); break;
    }
#undef MSDA_ROTARY_GO
    return cudaGetLastError();
}
template <typename T>
cudaError_t launch_rotary_weight(const float* partial, int n, int D, void* dwq, void* dwk, cudaStream_t st) {
    msda_rotary_weight_kernel<T><<<(2 * D + 31) / 32, 1024, 0, st>>>(partial, n, D, static_cast<T*>(dwq),
                                                                   static_cast<T*>(dwk));
    return cudaGetLastError();
}
#define MSDA_ROTARY_INSTANCES(T)                                                                                     \
    template cudaError_t launch_rotary<T>(const RotaryArgs&, int, bool, bool, int, bool, unsigned, size_t,           \
                                          cudaStream_t);                                                             \
    template cudaError_t launch_rotary_weight<T>(const float*, int, int, void*, void*, cudaStream_t);
#endif

}  // namespace msda
