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
// What bounds it: memory.  Every element is read once (twice in the backward:
// x and dy) and written once; all heads of a token share its angles, so a
// block first works out cos and sin of a chunk of tokens into shared memory
// (one sincos a token and pair, against (M + N) * 2 elements that use it) and
// then streams the rows.  A row is taken by a group of lanes, 16 bytes a load;
// a lane owns both halves of its pairs, so the rotation needs no exchange and
// the row's sums take log2(lanes) shuffles.  The weights' gradients stay in
// registers over all rows of a lane, then go through one partial row a block
// and a second kernel that adds the partials in a fixed order: no atomics.
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
    int T;              // tokens a chunk
    int chunks_per_b;
    long long chunks;
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

// cos and sin of p * f.  The product of two binary32 numbers is held exactly
// as hi + lo; hi is brought near [-pi, pi] by subtracting n times 2 pi, taken
// as three binary32 parts (Cody and Waite's reduction): the first subtraction
// is exact for |hi| < 2^23 (both sides are multiples of the smaller one's last
// place and the difference is below 4), so the angle is off by about 2^-24 in
// all whatever the position.  Larger products, and integer positions that
// binary32 does not hold, take the same reduction in binary64.
__device__ __forceinline__ void angle_cos_sin(double p64, float p, bool exact32, float f, float* c, float* s) {
    float r;
    const float hi = p * f;
    if (exact32 && fabsf(hi) < 8388608.f) {
        const float lo = fmaf(p, f, -hi);
        const float n = rintf(hi * 0.15915494309189535f);
        r = fmaf(-n, 6.2831854820251465f, hi);      // binary32 nearest to 2 pi
        r = fmaf(-n, -1.7484555314695172e-07f, r);  // the rest of 2 pi
        r += lo;
    } else {
        // up to 2^53 the product keeps its fraction; 2 pi in two binary64 parts
        const double t = p64 * (double)f;
        const double n = rint(t * 0.15915494309189535);
        double d = fma(-n, 6.283185307179586, t);
        d = fma(-n, 2.4492935982947064e-16, d);
        r = (float)d;
    }
    sincosf(r, s, c);
}

// cos / sin table of the chunk's tokens: [tokens][P] (cos, sin)
__device__ __forceinline__ void rotary_table(const RotaryArgs& a, long long b, int s0, int nt, float2* table) {
    for (int i = threadIdx.x; i < nt * a.P; i += kRotaryThreads) {
        const int t = i / a.P, j = i - t * a.P;
        int ax = 0;
        while (ax < a.A - 1 && j >= a.axis_end[ax]) ++ax;
        const long long at = b * a.pos_sb + (long long)(s0 + t) * a.A + ax;
        double p64;
        float p;
        bool exact32 = true;
        if (a.pos_type == 0) {
            p = static_cast<const float*>(a.pos)[at];
            p64 = p;
        } else {
            const long long v = a.pos_type == 1 ? (long long)static_cast<const int*>(a.pos)[at]
                                                : static_cast<const long long*>(a.pos)[at];
            p = (float)v;
            p64 = (double)v;
            exact32 = v > -16777217ll && v < 16777217ll;
        }
        float c, s;
        angle_cos_sin(p64, p, exact32, a.freq[j], &c, &s);
        table[i] = make_float2(c, s * a.sign);
    }
}

enum { ROT_SCALAR = 0, ROT_HALVES = 1, ROT_INTERLEAVED = 2 };

// What a lane holds of a row: up to two vectors of V channels at channel c0
// and c1 (c1 < 0: absent); HALVES: c1 = c0 + P when the item is rotated.
template <int V>
struct RotaryItem {
    int c0, c1;
    bool on, turned;
};

template <int MODE, int V>
__device__ __forceinline__ RotaryItem<V> rotary_item(int l, int D, int P) {
    RotaryItem<V> it;
    if constexpr (MODE == ROT_HALVES) {
        const int np = P / V;
        it.turned = l < np;
        it.c0 = it.turned ? l * V : (l + np) * V;
        it.c1 = it.turned ? l * V + P : -1;
        it.on = it.c0 < D;
    } else {
        it.turned = true;
        it.c0 = l * V;
        it.c1 = -1;
        it.on = it.c0 < D;
    }
    return it;
}

// z (the lane's channels: V of the first vector, V of the second) turned by
// the token's angles; `inv` turns back (dz = R^T dy).
template <int MODE, int V>
__device__ __forceinline__ void rotary_turn(float* z, const RotaryItem<V>& it, const float2* tab, int P, bool inv) {
    if constexpr (MODE == ROT_HALVES) {
        if (it.turned) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float2 cs = tab[it.c0 + i];
                const float s = inv ? -cs.y : cs.y;
                const float u = z[i], v = z[V + i];
                z[i] = u * cs.x - v * s;
                z[V + i] = v * cs.x + u * s;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const int j = (it.c0 + i) >> 1;
            if (j < P) {
                const float2 cs = tab[j];
                const float s = inv ? -cs.y : cs.y;
                const float u = z[i], v = z[i + 1];
                z[i] = u * cs.x - v * s;
                z[i + 1] = v * cs.x + u * s;
            }
        }
    }
}

// The chunk's rows of one tensor, vector form.  LG = log2 of the lanes a row.
template <typename T, int MODE, bool NORM, bool BWD>
__device__ __forceinline__ void rotary_rows_vec(const RotaryArgs& a, const RotaryTensor& t, int lg, long long b, int s0,
                                                int nt, const float2* table, float* dw) {
    constexpr int V = Vec16<T>::N;
    constexpr int W = MODE == ROT_HALVES ? 2 * V : V;
    constexpr int U = BWD ? 1 : 2;  // rows in flight a lane (measured: two hide the loads' latency; the backward has two tensors in flight already)
    const int lane_row = threadIdx.x & ((1 << lg) - 1);
    const int group = threadIdx.x >> lg;
    const int groups = kRotaryThreads >> lg;
    const RotaryItem<V> it = rotary_item<MODE, V>(lane_row, a.D, a.P);
    const T* x = static_cast<const T*>(t.x) + b * t.sb + (long long)s0 * t.ss;
    const long long dense0 = (b * a.S + s0) * (long long)t.heads * a.D;
    T* y = static_cast<T*>(t.y) + dense0;
    const T* dy = BWD ? static_cast<const T*>(t.dy) + dense0 : nullptr;
    float w[NORM ? W : 1];
    if constexpr (NORM) {
        const T* wp = static_cast<const T*>(t.w);
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0.f;
        if (it.on) {
            Vec16<T>::load(wp + it.c0, w);
            if (MODE == ROT_HALVES && it.c1 >= 0) Vec16<T>::load(wp + it.c1, w + (MODE == ROT_HALVES ? V : 0));
        }
    }
    const int rows = nt * t.heads;
    int tok[U], head[U];
    // rows group, group + groups, ... : token and head advance without a division
    const int dt = groups / t.heads, dh = groups - dt * t.heads;
    {
        int tk = group / t.heads, hd = group - tk * t.heads;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            tok[u] = tk, head[u] = hd;
            tk += dt, hd += dh;
            if (hd >= t.heads) hd -= t.heads, ++tk;
        }
    }
    // every lane of a warp takes the same number of turns: the shuffles below need all of them
    const int first_in_warp = (threadIdx.x & ~31) >> lg;
    for (int r0 = 0; first_in_warp + r0 < rows; r0 += groups * U) {
        float xv[U][W], gv[BWD ? W : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < W; ++i) xv[u][i] = 0.f;
            if (it.on && tok[u] < nt) {
                const T* p = x + (long long)tok[u] * t.ss + (long long)head[u] * t.sh;
                Vec16<T>::load(p + it.c0, xv[u]);
                if (MODE == ROT_HALVES && it.c1 >= 0) Vec16<T>::load(p + it.c1, xv[u] + (MODE == ROT_HALVES ? V : 0));
            }
        }
        if constexpr (BWD) {
#pragma unroll
            for (int i = 0; i < W; ++i) gv[i] = 0.f;
            if (it.on && tok[0] < nt) {
                const T* p = dy + ((long long)tok[0] * t.heads + head[0]) * a.D;
                Vec16<T>::load(p + it.c0, gv);
                if (MODE == ROT_HALVES && it.c1 >= 0) Vec16<T>::load(p + it.c1, gv + (MODE == ROT_HALVES ? V : 0));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float r = 1.f;
            if constexpr (NORM) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < W; ++i) ss = fmaf(xv[u][i], xv[u][i], ss);
                for (int o = (1 << lg) >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                r = rsqrtf(ss * a.inv_d + a.eps);
            }
            const bool live = it.on && tok[u] < nt;
            const float2* tab = table + (live ? tok[u] : 0) * a.P;
            if constexpr (!BWD) {
                if constexpr (NORM) {
#pragma unroll
                    for (int i = 0; i < W; ++i) xv[u][i] = xv[u][i] * r * w[i];
                }
                if (live) {
                    rotary_turn<MODE, V>(xv[u], it, tab, a.P, false);
                    T* p = y + ((long long)tok[u] * t.heads + head[u]) * a.D;
                    Vec16<T>::store(p + it.c0, xv[u]);
                    if (MODE == ROT_HALVES && it.c1 >= 0) Vec16<T>::store(p + it.c1, xv[u] + (MODE == ROT_HALVES ? V : 0));
                }
            } else {
                if (live) rotary_turn<MODE, V>(gv, it, tab, a.P, true);
                float dot = 0.f;
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    xv[u][i] *= r;  // n
                    dw[i] = fmaf(gv[i], xv[u][i], dw[i]);
                    gv[i] *= w[i];
                    dot = fmaf(gv[i], xv[u][i], dot);
                }
                for (int o = (1 << lg) >> 1; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                dot *= a.inv_d;
                if (live) {
#pragma unroll
                    for (int i = 0; i < W; ++i) gv[i] = r * fmaf(-xv[u][i], dot, gv[i]);
                    T* p = y + ((long long)tok[u] * t.heads + head[u]) * a.D;
                    Vec16<T>::store(p + it.c0, gv);
                    if (MODE == ROT_HALVES && it.c1 >= 0) Vec16<T>::store(p + it.c1, gv + (MODE == ROT_HALVES ? V : 0));
                }
            }
        }
        // U * groups rows on
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int k = 0; k < U; ++k) {
                tok[u] += dt, head[u] += dh;
                if (head[u] >= t.heads) head[u] -= t.heads, ++tok[u];
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

// Persistent over chunks of T tokens of one batch item.  Shared memory:
// float2[T][P], reused as float[8][D] for the weights' gradients at the end.
template <typename T, int MODE, bool NORM, bool BWD>
__global__ void __launch_bounds__(kRotaryThreads) msda_rotary_kernel(const RotaryArgs a, int lg, bool inter) {
    extern __shared__ __align__(16) unsigned char rotary_smem[];
    float2* table = reinterpret_cast<float2*>(rotary_smem);
    constexpr int V = Vec16<T>::N;
    constexpr int W = MODE == ROT_SCALAR ? 16 : MODE == ROT_HALVES ? 2 * V : V;
    float dw[2][BWD ? W : 1];
    if constexpr (BWD) {
#pragma unroll
        for (int i = 0; i < W; ++i) dw[0][i] = dw[1][i] = 0.f;
    }
    for (long long ch = blockIdx.x; ch < a.chunks; ch += gridDim.x) {
        const long long b = ch / a.chunks_per_b;
        const int s0 = (int)(ch - b * a.chunks_per_b) * a.T;
        const int nt = min(a.T, a.S - s0);
        __syncthreads();  // the table of the chunk before is no longer read
        rotary_table(a, b, s0, nt, table);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (a.t[k].heads == 0) continue;
            if constexpr (MODE == ROT_SCALAR)
                rotary_rows_scalar<T, NORM, BWD>(a, a.t[k], inter, b, s0, nt, table, dw[k]);
            else
                rotary_rows_vec<T, MODE, NORM, BWD>(a, a.t[k], lg, b, s0, nt, table, dw[k]);
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
            for (int c = lane; c < a.D; c += 32) red[warp * a.D + c] = 0.f;
            __syncwarp();
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
                const RotaryItem<V> it = rotary_item<MODE, V>(lane & ((1 << lg) - 1), a.D, a.P);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    float v = dw[k][i];
                    for (int o = 1 << lg; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                    const int c = i < V ? it.c0 + i : it.c1 + i - V;
                    if (lane < (1 << lg) && it.on && (i < V || it.c1 >= 0)) red[warp * a.D + c] = v;
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
__global__ void __launch_bounds__(256) msda_rotary_weight_kernel(const float* partial, int n, int D, T* dwq, T* dwk) {
    __shared__ float red[8][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
    float v = 0.f;
    if (col < 2 * D)
        for (int i = part; i < n; i += 8) v += partial[(long long)i * 2 * D + col];
    red[part][threadIdx.x & 31] = v;
    __syncthreads();
    if (part == 0 && col < 2 * D) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += red[i][threadIdx.x & 31];
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
    msda_rotary_weight_kernel<T><<<(2 * D + 31) / 32, 256, 0, st>>>(partial, n, D, static_cast<T*>(dwq),
                                                                   static_cast<T*>(dwk));
    return cudaGetLastError();
}
#define MSDA_ROTARY_INSTANCES(T)                                                                                     \
    template cudaError_t launch_rotary<T>(const RotaryArgs&, int, bool, bool, int, bool, unsigned, size_t,           \
                                          cudaStream_t);                                                             \
    template cudaError_t launch_rotary_weight<T>(const float*, int, int, void*, void*, cudaStream_t);
#endif

}  // namespace msda
