// msda_attention_simt.cuh -- softmax attention and its gradients on the FMA
// pipe: every dtype, every D up to 128, every alignment.
//
// binary32 tensors run here where the tensor cores do not take them in pieces
// (more than 64 channels, small calls, values beyond the pieces' range), and
// 16-bit tensors whose rows or strides are not made of 16-byte vectors.
//
// A block takes 64 rows against tiles of 64 others; 128 threads, each 8 x 4
// scores and 8 x D/16 outputs in registers.  Per 4 channels a thread reads
// 8 + 4 vectors of shared memory for 128 FMA: 16 shared-memory wavefronts a
// warp against 32 FMA-pipe cycles, so the FMA pipe bounds it.  Rows are padded
// by 4 floats: the 16 lanes that read 16 rows at one channel then hit each
// bank once a phase.
#pragma once

#include "msda_attention.cuh"
#include "msda_host.cuh"

namespace msda {

constexpr int kSimtThreads = 128;
constexpr int kSimtRows = 64;
// blocks an SM that registers leave room for (accumulators grow with DP)
constexpr int simt_blocks(int dp) { return dp <= 64 ? 3 : 2; }

template <typename T>
__device__ __forceinline__ float attn_f32(T v) { return (float)v; }
template <typename T>
__device__ __forceinline__ T attn_round(float v);
template <>
__device__ __forceinline__ float attn_round<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half attn_round<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 attn_round<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// 64 rows of D channels (rows at or above `rows`, and those `alive` says no
// for, as zeros) into dst[64][DP + 4]; channels from D to DP are zeros.
// binary32 rows of whole 16-byte vectors go by asynchronous copies, which a
// caller issues as soon as a buffer is free and waits for (simt_landed) only
// before its use: with plain loads the FMA pipe was busy 28 % of the time.
template <typename T, int DP>
__device__ __forceinline__ void simt_load(float* dst, const T* src, long long stride, int rows, int D, bool vec,
                                          const uint8_t* alive) {
    constexpr int LD = DP + 4;
    if constexpr (sizeof(T) == 4) {
        if (vec) {
            for (int i = threadIdx.x; i < kSimtRows * (DP / 4); i += kSimtThreads) {
                const int r = i / (DP / 4), c = (i - r * (DP / 4)) * 4;
                const bool in = r < rows && c < D && (!alive || alive[r]);
                const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst + r * LD + c);
                // a source size of 0 writes zeros and reads nothing
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to),
                             "l"(in ? (const void*)(src + r * stride + c) : (const void*)src), "r"(in ? 16 : 0)
                             : "memory");
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            return;
        }
    }
    for (int i = threadIdx.x; i < kSimtRows * DP; i += kSimtThreads) {
        const int r = i / DP, c = i - r * DP;
        dst[r * LD + c] = r < rows && c < D && (!alive || alive[r]) ? attn_f32(src[r * stride + c]) : 0.f;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// all but the last `N` loads have landed, for every thread of the block
template <int N>
__device__ __forceinline__ void simt_landed() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
    __syncthreads();
}

// acc[i][c] += sum_d A[ty*8+i][d] B[tx+16c][d]
template <int DP>
__device__ __forceinline__ void simt_nt(float (&acc)[8][4], const float* A, const float* B, int tx, int ty) {
    constexpr int LD = DP + 4;
#pragma unroll 1
    for (int d = 0; d < DP; d += 4) {
        float4 a[8], b[4];
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = *reinterpret_cast<const float4*>(A + (ty * 8 + i) * LD + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = *reinterpret_cast<const float4*>(B + (tx + 16 * c) * LD + d);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                acc[i][c] = fmaf(a[i].x, b[c].x, acc[i][c]);
                acc[i][c] = fmaf(a[i].y, b[c].y, acc[i][c]);
                acc[i][c] = fmaf(a[i].z, b[c].z, acc[i][c]);
                acc[i][c] = fmaf(a[i].w, b[c].w, acc[i][c]);
            }
    }
}

constexpr int kSimtLdP = 64 + 4;

// acc[i][c] += sum_k P[ty*8+i][k] X[k][tx+16c]
template <int DP>
__device__ __forceinline__ void simt_nn(float (&acc)[8][DP / 16], const float* P, const float* X, int tx, int ty) {
    constexpr int LD = DP + 4;
#pragma unroll 1
    for (int k = 0; k < 64; k += 4) {
        float4 p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = *reinterpret_cast<const float4*>(P + (ty * 8 + i) * kSimtLdP + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            float x[DP / 16];
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) x[c] = X[(k + kk) * LD + tx + 16 * c];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float pv = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
#pragma unroll
                for (int c = 0; c < DP / 16; ++c) acc[i][c] = fmaf(pv, x[c], acc[i][c]);
            }
        }
    }
}

// acc[i][c] += sum_q P[q][ty*8+i] X[q][tx+16c]
template <int DP>
__device__ __forceinline__ void simt_tn(float (&acc)[8][DP / 16], const float* P, const float* X, int tx, int ty) {
    constexpr int LD = DP + 4;
#pragma unroll 4
    for (int q = 0; q < 64; ++q) {
        const float4 p0 = *reinterpret_cast<const float4*>(P + q * kSimtLdP + ty * 8);
        const float4 p1 = *reinterpret_cast<const float4*>(P + q * kSimtLdP + ty * 8 + 4);
        const float p[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
            const float x = X[q * LD + tx + 16 * c];
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i][c] = fmaf(p[i], x, acc[i][c]);
        }
    }
}

// Words of a row's 64 keys from j0 on (a multiple of 64) in the mask's bits.
__device__ __forceinline__ uint2 simt_bits(const AttentionArgs& a, int b, int m, int q, int j0) {
    return *reinterpret_cast<const uint2*>(a.bits + b * a.bits_sb + m * a.bits_sh + (long long)q * a.W + (j0 >> 5));
}
// Whether the mask leaves any pair of the tile (the whole block asks; also a barrier).
__device__ __forceinline__ bool simt_tile_seen(const AttentionArgs& a, int b, int m, int q0, int j0) {
    bool any = false;
    if (threadIdx.x < 64 && q0 + (int)threadIdx.x < a.Q) {
        const uint2 w = simt_bits(a, b, m, q0 + threadIdx.x, j0);
        any = (w.x | w.y) != 0;
    }
    return __syncthreads_or(any);
}

// Scores in log2 units of the block's rows q0 + ty*8 + i and keys j0 + tx + 16c; -inf where the pair takes no part.
__device__ __forceinline__ void simt_mask(float (&s)[8][4], const AttentionArgs& a, int b, int m, int q0, int j0, int tx,
                                          int ty) {
    const uint8_t* km = a.key_mask ? a.key_mask + b * a.km_sb + (m / a.G) * a.km_sh : nullptr;
    bool in[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int j = j0 + tx + 16 * c;
        in[c] = j < a.S && (!km || km[j]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int q = q0 + ty * 8 + i;
        uint2 w = make_uint2(~0u, ~0u);
        if (a.bits && q < a.Q) w = simt_bits(a, b, m, q, j0);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            bool ok = in[c] && q < a.Q && (((c < 2 ? w.x : w.y) >> (tx + 16 * (c & 1))) & 1u);
            if (a.causal) ok = ok && j0 + tx + 16 * c <= q + (a.S - a.Q);
            s[i][c] = ok ? s[i][c] * a.c2 : -attn_inf();
        }
    }
}

__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Tiles of 64 keys that rows q0 .. q0+63 can see.
__device__ __forceinline__ int simt_key_tiles(const AttentionArgs& a, int q0) {
    long long last = a.S;
    if (a.causal) {
        const long long see = (long long)min(q0 + kSimtRows, a.Q) + (a.S - a.Q);
        last = see < 0 ? 0 : see < a.S ? see : a.S;
    }
    return (int)((last + 63) / 64);
}

// Statistics of a head's rows from q0 on (a multiple of 64) in tiles of rw.rt rows.
__device__ __forceinline__ long long simt_stat(const AttentionRows& rw, long long head, int q0) {
    return (head * rw.tiles + q0 / rw.rt) * 2 * rw.rt + q0 % rw.rt;
}

// binary32 behind the tensor cores' kernels, which did the work unless a value was not fit for them
__device__ __forceinline__ bool simt_done(const AttentionArgs& a) { return a.odd && !*a.odd; }

// Forward: running maximum m and sum l of each row, O rescaled when m grows.
template <typename T, int DP>
__global__ void __launch_bounds__(kSimtThreads, simt_blocks(DP)) msda_attention_simt_kernel(const AttentionArgs a, bool vec) {
    extern __shared__ __align__(16) float simt_smem[];
    if (simt_done(a)) return;
    constexpr int LD = DP + 4;
    float* Qs = simt_smem;
    float* Ks = Qs + kSimtRows * LD;
    float* Vs = Ks + kSimtRows * LD;
    float* Ps = Vs + kSimtRows * LD;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int qtiles = (a.Q + kSimtRows - 1) / kSimtRows;
    long long id = blockIdx.x;
    const int split = (int)(id % a.splits);
    id /= a.splits;
    const int q0 = (int)(id % qtiles) * kSimtRows;
    id /= qtiles;
    const int m = (int)(id % a.M), b = (int)(id / a.M), n = m / a.G;
    const T* q = static_cast<const T*>(a.q) + b * a.q_sb + m * a.q_sh + q0 * a.q_ss;
    const T* k = static_cast<const T*>(a.k) + b * a.k_sb + n * a.k_sh;
    const T* v = static_cast<const T*>(a.v) + b * a.v_sb + n * a.v_sh;
    const uint8_t* km = a.key_mask ? a.key_mask + b * a.km_sb + n * a.km_sh : nullptr;
    simt_load<T, DP>(Qs, q, a.q_ss, a.Q - q0, a.D, vec, nullptr);
    float o[8][DP / 16], mx[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        mx[i] = -attn_inf(), l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) o[i][c] = 0.f;
    }
    const int t0 = split * a.tiles_per_split;
    const int t1 = min(simt_key_tiles(a, q0), t0 + a.tiles_per_split);
    auto fetch = [&](float* to, const T* from, long long stride, int t) {
        simt_load<T, DP>(to, from + t * 64 * stride, stride, a.S - t * 64, a.D, vec, km ? km + t * 64 : nullptr);
    };
    auto seen_from = [&](int t) {  // the next tile that the mask leaves a pair of
        if (a.bits)
            while (t < t1 && !simt_tile_seen(a, b, m, q0, t * 64)) ++t;
        return t;
    };
    int t = seen_from(t0);
    if (t < t1) {
        fetch(Ks, k, a.k_ss, t);
        fetch(Vs, v, a.v_ss, t);
    }
    while (t < t1) {
        const int j0 = t * 64, next = seen_from(t + 1);
        simt_landed<1>();
        float s[8][4] = {};
        simt_nt<DP>(s, Qs, Ks, tx, ty);
        simt_mask(s, a, b, m, q0, j0, tx, ty);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float top = fmaxf(mx[i], half_warp_max(fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]))));
            const float ref = top == -attn_inf() ? 0.f : top;  // a row that has seen nothing yet
            const float f = exp2f(mx[i] - ref);
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float p = exp2f(s[i][c] - ref);
                sum += p;
                Ps[(ty * 8 + i) * kSimtLdP + tx + 16 * c] = p;
            }
            l[i] = l[i] * f + half_warp_sum(sum);
            mx[i] = top;
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) o[i][c] *= f;
        }
        __syncthreads();  // keys read, P written
        if (next < t1) {
            fetch(Ks, k, a.k_ss, next);
            simt_landed<1>();
        } else {
            simt_landed<0>();
        }
        simt_nn<DP>(o, Ps, Vs, tx, ty);
        __syncthreads();
        if (next < t1) fetch(Vs, v, a.v_ss, next);
        t = next;
    }
    simt_landed<0>();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int qi = q0 + ty * 8 + i;
        if (qi >= a.Q) continue;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        const float l2 = l[i] == 0.f ? -attn_inf() : mx[i] + log2f(l[i]);
        const long long row = ((long long)b * a.M + m) * a.Q + qi;
        if (a.splits > 1) {
            const long long at = (long long)split * a.B * a.M * a.Q + row;
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) {
                const int d = tx + 16 * c;
                if (d < a.D) a.part_o[at * a.D + d] = o[i][c] * inv;
            }
            if (tx == 0) a.part_lse[at] = l2;
        } else {
            T* out = static_cast<T*>(a.out) + (((long long)b * a.Q + qi) * a.M + m) * a.D;
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) {
                const int d = tx + 16 * c;
                if (d < a.D) out[d] = attn_round<T>(o[i][c] * inv);
            }
            if (tx == 0) a.lse[row] = l2 * kLn2;
        }
    }
}

// p and ds of a tile: s in, on return s = p and dp = p (dp - delta), each 0
// where the pair takes no part.  Rows' statistics: l2 = -lse (-inf: no part), dl = -delta.
__device__ __forceinline__ void simt_prob_grad(float (&s)[8][4], float (&dp)[8][4], const float* l2, const float* dl) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float p = s[i][c] == -attn_inf() ? 0.f : exp2f(s[i][c] + l2[i]);
            s[i][c] = p;
            dp[i][c] = p == 0.f ? 0.f : p * (dp[i][c] + dl[i]);
        }
}

// Gradients of 64 keys and values of one key head: over all queries of the
// heads that share it, so the sums over shared heads stay in registers.
template <typename T, int DP>
__global__ void __launch_bounds__(kSimtThreads, simt_blocks(DP)) msda_attention_simt_grad_key_kernel(const AttentionArgs a,
                                                                                    const AttentionRows rw, bool vec) {
    extern __shared__ __align__(16) float simt_smem[];
    if (simt_done(a)) return;
    constexpr int LD = DP + 4;
    float* Ks = simt_smem;
    float* Vs = Ks + kSimtRows * LD;
    float* Qs = Vs + kSimtRows * LD;
    float* Gs = Qs + kSimtRows * LD;
    float* Ps = Gs + kSimtRows * LD;  // p, then ds
    uint8_t* live = reinterpret_cast<uint8_t*>(Ps + kSimtRows * kSimtLdP);  // rows of the query tile that take part
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int ktiles = (a.S + 63) / 64;
    long long id = blockIdx.x;
    const int j0 = (int)(id % ktiles) * 64;
    id /= ktiles;
    const int n = (int)(id % a.N), b = (int)(id / a.N);
    const T* k = static_cast<const T*>(a.k) + b * a.k_sb + n * a.k_sh + j0 * a.k_ss;
    const T* v = static_cast<const T*>(a.v) + b * a.v_sb + n * a.v_sh + j0 * a.v_ss;
    const uint8_t* km = a.key_mask ? a.key_mask + b * a.km_sb + n * a.km_sh + j0 : nullptr;
    simt_load<T, DP>(Ks, k, a.k_ss, a.S - j0, a.D, vec, km);
    simt_load<T, DP>(Vs, v, a.v_ss, a.S - j0, a.D, vec, km);
    float dk[8][DP / 16] = {}, dv[8][DP / 16] = {};
    // causal: queries below j0 - (S - Q) see none of these keys
    long long first = a.causal ? (long long)j0 - (a.S - a.Q) : 0;
    if (first < 0) first = 0;
    const int qt0 = (int)(first / 64), qts = (a.Q + 63) / 64, per = qts > qt0 ? qts - qt0 : 0, total = a.G * per;
    // step x: query tile qt0 + x % per of head x / per; the next one that the mask leaves a pair of
    auto seen_from = [&](int x) {
        if (a.bits)
            while (x < total && !simt_tile_seen(a, b, n * a.G + x / per, (qt0 + x % per) * 64, j0)) ++x;
        return x;
    };
    auto stat_at = [&](int x) { return simt_stat(rw, (long long)b * rw.heads + n * a.G + x / per, (qt0 + x % per) * 64); };
    // rows that take no part are cleared: their flags are written a tile ahead of the copies that ask for them
    auto flags = [&](int x) {
        if (threadIdx.x < 64) live[threadIdx.x] = a.row_l2[stat_at(x) + threadIdx.x] != -attn_inf();
    };
    auto fetch_q = [&](int x) {
        const int m = n * a.G + x / per, q0 = (qt0 + x % per) * 64;
        simt_load<T, DP>(Qs, static_cast<const T*>(a.q) + b * a.q_sb + m * a.q_sh + q0 * a.q_ss, a.q_ss, a.Q - q0, a.D, vec, live);
    };
    auto fetch_g = [&](int x) {
        const int m = n * a.G + x / per, q0 = (qt0 + x % per) * 64;
        simt_load<T, DP>(Gs, static_cast<const T*>(a.dout) + (((long long)b * a.Q + q0) * a.M + m) * a.D,
                         (long long)a.M * a.D, a.Q - q0, a.D, vec, live);
    };
    int x = seen_from(0);
    if (x < total) {
        flags(x);
        __syncthreads();
        fetch_g(x);
        fetch_q(x);
    }
    while (x < total) {
        const int m = n * a.G + x / per, q0 = (qt0 + x % per) * 64;
        const int next = seen_from(x + 1);
        simt_landed<1>();  // the gradient's rows (and K, V)
        float s[8][4] = {}, dp[8][4] = {}, l2[8], dl[8];
        simt_nt<DP>(dp, Gs, Vs, tx, ty);
        const long long at = stat_at(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) l2[i] = a.row_l2[at + ty * 8 + i], dl[i] = a.row_dl[at + ty * 8 + i];
        simt_landed<0>();
        if (next < total) flags(next);  // both tiles have landed: the old flags are done with
        simt_nt<DP>(s, Qs, Ks, tx, ty);
        simt_mask(s, a, b, m, q0, j0, tx, ty);
        simt_prob_grad(s, dp, l2, dl);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) Ps[(ty * 8 + i) * kSimtLdP + tx + 16 * c] = s[i][c];
        __syncthreads();
        simt_tn<DP>(dv, Ps, Gs, tx, ty);
        __syncthreads();
        if (next < total) fetch_g(next);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) Ps[(ty * 8 + i) * kSimtLdP + tx + 16 * c] = dp[i][c];
        __syncthreads();
        simt_tn<DP>(dk, Ps, Qs, tx, ty);
        __syncthreads();
        if (next < total) fetch_q(next);
        x = next;
    }
    simt_landed<0>();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int j = j0 + ty * 8 + i;
        if (j >= a.S) continue;
        const long long at = (((long long)b * a.S + j) * a.N + n) * a.D;
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
            const int d = tx + 16 * c;
            if (d < a.D) {
                static_cast<T*>(a.dk)[at + d] = attn_round<T>(dk[i][c] * a.scale);
                static_cast<T*>(a.dv)[at + d] = attn_round<T>(dv[i][c]);
            }
        }
    }
}

// Gradient of 64 queries of one head: over the keys that they see.
template <typename T, int DP>
__global__ void __launch_bounds__(kSimtThreads, simt_blocks(DP)) msda_attention_simt_grad_query_kernel(const AttentionArgs a,
                                                                                      const AttentionRows rw, bool vec) {
    extern __shared__ __align__(16) float simt_smem[];
    if (simt_done(a)) return;
    constexpr int LD = DP + 4;
    float* Qs = simt_smem;
    float* Gs = Qs + kSimtRows * LD;
    float* Ks = Gs + kSimtRows * LD;
    float* Vs = Ks + kSimtRows * LD;
    float* Ps = Vs + kSimtRows * LD;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int qtiles = (a.Q + 63) / 64;
    long long id = blockIdx.x;
    const int q0 = (int)(id % qtiles) * 64;
    id /= qtiles;
    const int m = (int)(id % a.M), b = (int)(id / a.M), n = m / a.G;
    const T* k = static_cast<const T*>(a.k) + b * a.k_sb + n * a.k_sh;
    const T* v = static_cast<const T*>(a.v) + b * a.v_sb + n * a.v_sh;
    const uint8_t* km = a.key_mask ? a.key_mask + b * a.km_sb + n * a.km_sh : nullptr;
    simt_load<T, DP>(Qs, static_cast<const T*>(a.q) + b * a.q_sb + m * a.q_sh + q0 * a.q_ss, a.q_ss, a.Q - q0, a.D, vec,
                     nullptr);
    simt_load<T, DP>(Gs, static_cast<const T*>(a.dout) + (((long long)b * a.Q + q0) * a.M + m) * a.D,
                     (long long)a.M * a.D, a.Q - q0, a.D, vec, nullptr);
    float l2[8], dl[8], dq[8][DP / 16] = {};
    const long long at0 = simt_stat(rw, (long long)b * rw.heads + m, q0);
#pragma unroll
    for (int i = 0; i < 8; ++i) l2[i] = a.row_l2[at0 + ty * 8 + i], dl[i] = a.row_dl[at0 + ty * 8 + i];
    const int tiles = simt_key_tiles(a, q0);
    auto fetch = [&](float* to, const T* from, long long stride, int t) {
        simt_load<T, DP>(to, from + t * 64 * stride, stride, a.S - t * 64, a.D, vec, km ? km + t * 64 : nullptr);
    };
    auto seen_from = [&](int t) {
        if (a.bits)
            while (t < tiles && !simt_tile_seen(a, b, m, q0, t * 64)) ++t;
        return t;
    };
    int t = seen_from(0);
    if (t < tiles) {
        fetch(Vs, v, a.v_ss, t);
        fetch(Ks, k, a.k_ss, t);
    }
    while (t < tiles) {
        const int j0 = t * 64, next = seen_from(t + 1);
        simt_landed<1>();
        float s[8][4] = {}, dp[8][4] = {};
        simt_nt<DP>(dp, Gs, Vs, tx, ty);
        simt_landed<0>();
        if (next < tiles) fetch(Vs, v, a.v_ss, next);
        simt_nt<DP>(s, Qs, Ks, tx, ty);
        simt_mask(s, a, b, m, q0, j0, tx, ty);
        simt_prob_grad(s, dp, l2, dl);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) Ps[(ty * 8 + i) * kSimtLdP + tx + 16 * c] = dp[i][c];
        __syncthreads();
        simt_nn<DP>(dq, Ps, Ks, tx, ty);
        __syncthreads();
        if (next < tiles) fetch(Ks, k, a.k_ss, next);
        t = next;
    }
    simt_landed<0>();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int qi = q0 + ty * 8 + i;
        if (qi >= a.Q) continue;
        T* out = static_cast<T*>(a.dq) + (((long long)b * a.Q + qi) * a.M + m) * a.D;
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
            const int d = tx + 16 * c;
            if (d < a.D) out[d] = attn_round<T>(dq[i][c] * a.scale);
        }
    }
}

// Joins the rows of a split key axis: out = sum_i 2^(lse_i - lse) o_i.  A block
// a row, each warp every fourth part (one warp for 57 parts took 16 us), then
// the warps' sums in a fixed order.
template <typename T>
__global__ void __launch_bounds__(128) msda_attention_join_kernel(const AttentionArgs a) {
    __shared__ float part[4][kAttnMaxChannels + 1];
    const long long rows = (long long)a.B * a.M * a.Q, row = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float top = -attn_inf();
    for (int i = lane; i < a.splits; i += 32) {
        const float x = a.part_lse[i * rows + row];
        top = x != x ? x : fmaxf(top, x);
    }
    for (int o = 16; o > 0; o >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, top, o);
        top = x != x ? x : top != top ? top : fmaxf(top, x);
    }
    const float ref = top == -attn_inf() ? 0.f : top;
    float sum = 0.f, o[kAttnMaxChannels / 32] = {};
#pragma unroll 4
    for (int i = warp; i < a.splits; i += 4) {
        const float w = exp2f(a.part_lse[i * rows + row] - ref);
        sum += w;
        const float* p = a.part_o + (i * rows + row) * a.D;
#pragma unroll
        for (int c = 0; c < kAttnMaxChannels / 32; ++c)
            if (lane + 32 * c < a.D) o[c] = fmaf(w, p[lane + 32 * c], o[c]);
    }
#pragma unroll
    for (int c = 0; c < kAttnMaxChannels / 32; ++c) part[warp][lane + 32 * c] = o[c];
    if (lane == 0) part[warp][kAttnMaxChannels] = sum;
    __syncthreads();
    if (warp != 0) return;
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) sum += part[w][kAttnMaxChannels];
#pragma unroll
    for (int c = 0; c < kAttnMaxChannels / 32; ++c) {
        o[c] = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) o[c] += part[w][lane + 32 * c];
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const long long bm = row / a.Q;
    const int q = (int)(row - bm * a.Q);
    const long long b = bm / a.M;
    const int m = (int)(bm - b * a.M);
    T* out = static_cast<T*>(a.out) + ((b * a.Q + q) * a.M + m) * a.D;
#pragma unroll
    for (int c = 0; c < kAttnMaxChannels / 32; ++c)
        if (lane + 32 * c < a.D) out[lane + 32 * c] = attn_round<T>(o[c] * inv);
    if (lane == 0) a.lse[row] = sum == 0.f ? -attn_inf() : (ref + log2f(sum)) * kLn2;
}

// Statistics of the backward's rows: `off` - lse in log2 units (-inf where the
// row takes no part or is padding) and -<dout, out>.  A block takes a tile of
// rows of a head, eight lanes a row.
// With `top` (f16 on the tensor cores) also the largest squared norms of the
// rows of dout that take part, top[0], and, over tiles of 128 keys behind the
// rows' tiles, of the values that a query may see, top[1]; cleared before, taken
// as bits: non-negative numbers are in the order of their bits, so the order of
// the atomics changes nothing.
template <typename T>
__global__ void __launch_bounds__(256) msda_attention_prepare_kernel(const AttentionArgs a, const AttentionRows rw,
                                                                     const void* out_, const float* lse, float off,
                                                                     float* l2, float* top, bool vec) {
    const int vtiles = (a.S + 127) / 128;
    const long long tiles = (long long)a.B * rw.heads * rw.tiles;
    const long long units = tiles + (top ? (long long)a.B * a.N * vtiles : 0);
    const int lane = threadIdx.x & 7, group = threadIdx.x >> 3;
    float best_g = 0.f, best_v = 0.f;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const bool rows = u < tiles;
        const long long e = rows ? u : u - tiles;
        const int per = rows ? rw.tiles : vtiles, heads = rows ? rw.heads : a.N;
        const long long bh = e / per, b = bh / heads;
        const int t = (int)(e - bh * per), h = (int)(bh - b * heads), n = rows ? rw.rt : 128;
        for (int r = group; r < n; r += 32) {  // n is a multiple of 32: whole warps stay together
            const long long i = (long long)t * n + r;
            const T* g = nullptr;
            const T* o = nullptr;
            float x = 0.f;
            if (rows) {
                if (i < a.Q) {
                    x = lse[bh * a.Q + i];
                    if (x != -attn_inf()) {
                        const long long at = ((b * a.Q + i) * a.M + h) * a.D;
                        g = static_cast<const T*>(a.dout) + at;
                        o = static_cast<const T*>(out_) + at;
                    }
                }
            } else if (i < a.S && (!a.key_mask || a.key_mask[b * a.km_sb + h * a.km_sh + i])) {
                g = static_cast<const T*>(a.v) + b * a.v_sb + i * a.v_ss + h * a.v_sh;
            }
            float d = 0.f, gg = 0.f;
            if (g) {
                if (sizeof(T) == 2 && vec) {  // rows of whole 16-byte vectors
                    for (int c = lane * 8; c < a.D; c += 64) {
                        alignas(16) T gv[8], ov[8];
                        *reinterpret_cast<uint4*>(gv) = *reinterpret_cast<const uint4*>(g + c);
                        if (o) *reinterpret_cast<uint4*>(ov) = *reinterpret_cast<const uint4*>(o + c);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float y = attn_f32(gv[k]);
                            gg = fmaf(y, y, gg);
                            if (o) d = fmaf(y, attn_f32(ov[k]), d);
                        }
                    }
                } else {
                    for (int c = lane; c < a.D; c += 8) {
                        const float y = attn_f32(g[c]);
                        gg = fmaf(y, y, gg);
                        if (o) d = fmaf(y, attn_f32(o[c]), d);
                    }
                }
            }
            for (int s = 4; s > 0; s >>= 1) {
                d += __shfl_xor_sync(0xffffffffu, d, s);
                gg += __shfl_xor_sync(0xffffffffu, gg, s);
            }
            if (rows) {
                if (lane == 0) {
                    l2[u * 2 * n + r] = g ? off - x * kLog2e : -attn_inf();
                    l2[u * 2 * n + n + r] = g ? -d : 0.f;
                }
                best_g = gg > best_g || gg != gg ? gg : best_g;
            } else {
                best_v = gg > best_v || gg != gg ? gg : best_v;
            }
        }
    }
    if (top) {
        const unsigned ug = __reduce_max_sync(0xffffffffu, __float_as_uint(best_g) & 0x7fffffffu);
        const unsigned uv = __reduce_max_sync(0xffffffffu, __float_as_uint(best_v) & 0x7fffffffu);
        if ((threadIdx.x & 31) == 0 && ug) atomicMax(reinterpret_cast<unsigned*>(top), ug);
        if ((threadIdx.x & 31) == 0 && uv) atomicMax(reinterpret_cast<unsigned*>(top) + 1, uv);
    }
}

// Launches for dtype T (each in its own translation unit).
template <typename T>
cudaError_t launch_attention_simt(const AttentionArgs& a, bool vec, cudaStream_t st);
template <typename T>
cudaError_t launch_attention_simt_grad_key(const AttentionArgs& a, const AttentionRows& rw, bool vec, cudaStream_t st);
template <typename T>
cudaError_t launch_attention_simt_grad_query(const AttentionArgs& a, const AttentionRows& rw, bool vec, cudaStream_t st);
template <typename T>
cudaError_t launch_attention_join(const AttentionArgs& a, cudaStream_t st);
template <typename T>
cudaError_t launch_attention_prepare(const AttentionArgs& a, const AttentionRows& rw, const void* out, const float* lse,
                                     float off, float* l2, float* top, bool vec, cudaStream_t st);

#ifdef MSDA_ATTENTION_SIMT_INSTANTIATE
// head channels padded to a multiple of the 16 lanes that share a row
#define MSDA_SIMT_BY_D(D, GO) \
    do {                      \
        if ((D) <= 32) GO(32); \
        else if ((D) <= 48) GO(48); \
        else if ((D) <= 64) GO(64); \
        else if ((D) <= 96) GO(96); \
        else GO(128);         \
    } while (0)

template <typename T, int DP>
static cudaError_t simt_go(const AttentionArgs& a, bool vec, cudaStream_t st) {
    const size_t smem = (size_t)(3 * kSimtRows * (DP + 4) + kSimtRows * kSimtLdP) * 4;
    static SmemSeen seen;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(&msda_attention_simt_kernel<T, DP>), smem, seen);
    if (e != cudaSuccess) return e;
    const long long grid = (long long)a.B * a.M * ((a.Q + 63) / 64) * a.splits;
    msda_attention_simt_kernel<T, DP><<<(unsigned)grid, kSimtThreads, smem, st>>>(a, vec);
    return cudaGetLastError();
}
template <typename T, int DP>
static cudaError_t simt_grad_key_go(const AttentionArgs& a, const AttentionRows& rw, bool vec, cudaStream_t st) {
    const size_t smem = (size_t)(4 * kSimtRows * (DP + 4) + kSimtRows * kSimtLdP + 16) * 4;
    static SmemSeen seen;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(&msda_attention_simt_grad_key_kernel<T, DP>), smem, seen);
    if (e != cudaSuccess) return e;
    const long long grid = (long long)a.B * a.N * ((a.S + 63) / 64);
    msda_attention_simt_grad_key_kernel<T, DP><<<(unsigned)grid, kSimtThreads, smem, st>>>(a, rw, vec);
    return cudaGetLastError();
}
template <typename T, int DP>
static cudaError_t simt_grad_query_go(const AttentionArgs& a, const AttentionRows& rw, bool vec, cudaStream_t st) {
    const size_t smem = (size_t)(4 * kSimtRows * (DP + 4) + kSimtRows * kSimtLdP) * 4;
    static SmemSeen seen;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(&msda_attention_simt_grad_query_kernel<T, DP>), smem, seen);
    if (e != cudaSuccess) return e;
    const long long grid = (long long)a.B * a.M * ((a.Q + 63) / 64);
    msda_attention_simt_grad_query_kernel<T, DP><<<(unsigned)grid, kSimtThreads, smem, st>>>(a, rw, vec);
    return cudaGetLastError();
}
template <typename T>
cudaError_t launch_attention_simt(const AttentionArgs& a, bool vec, cudaStream_t st) {
#define MSDA_GO(DP) return simt_go<T, DP>(a, vec, st)
    MSDA_SIMT_BY_D(a.D, MSDA_GO);
#undef MSDA_GO
}
template <typename T>
cudaError_t launch_attention_simt_grad_key(const AttentionArgs& a, const AttentionRows& rw, bool vec, cudaStream_t st) {
#define MSDA_GO(DP) return simt_grad_key_go<T, DP>(a, rw, vec, st)
    MSDA_SIMT_BY_D(a.D, MSDA_GO);
#undef MSDA_GO
}
template <typename T>
cudaError_t launch_attention_simt_grad_query(const AttentionArgs& a, const AttentionRows& rw, bool vec, cudaStream_t st) {
#define MSDA_GO(DP) return simt_grad_query_go<T, DP>(a, rw, vec, st)
    MSDA_SIMT_BY_D(a.D, MSDA_GO);
#undef MSDA_GO
}
template <typename T>
cudaError_t launch_attention_join(const AttentionArgs& a, cudaStream_t st) {
    const long long rows = (long long)a.B * a.M * a.Q;
    msda_attention_join_kernel<T><<<(unsigned)rows, 128, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename T>
cudaError_t launch_attention_prepare(const AttentionArgs& a, const AttentionRows& rw, const void* out, const float* lse,
                                     float off, float* l2, float* top, bool vec, cudaStream_t st) {
    const long long units = (long long)a.B * rw.heads * rw.tiles + (top ? (long long)a.B * a.N * ((a.S + 127) / 128) : 0);
    const unsigned grid = (unsigned)(units < kPlanSms * 16 ? units : kPlanSms * 16);
    msda_attention_prepare_kernel<T><<<grid, 256, 0, st>>>(a, rw, out, lse, off, l2, top, vec);
    return cudaGetLastError();
}
#define MSDA_SIMT_INSTANCES(T)                                                                                          \
    template cudaError_t launch_attention_simt<T>(const AttentionArgs&, bool, cudaStream_t);                            \
    template cudaError_t launch_attention_simt_grad_key<T>(const AttentionArgs&, const AttentionRows&, bool, cudaStream_t); \
    template cudaError_t launch_attention_simt_grad_query<T>(const AttentionArgs&, const AttentionRows&, bool, cudaStream_t); \
    template cudaError_t launch_attention_join<T>(const AttentionArgs&, cudaStream_t);                                  \
    template cudaError_t launch_attention_prepare<T>(const AttentionArgs&, const AttentionRows&, const void*,           \
                                                     const float*, float, float*, float*, bool, cudaStream_t);
#endif

}  // namespace msda
