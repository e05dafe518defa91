// msda_attention_decode.cu -- softmax attention of a few query rows (queries
// times the heads that share a key head) over a long key axis, as one new token
// over a cache: one row in 16 bits, up to eight in binary32, D up to 128, rows
// of whole 16-byte vectors.
//
// What bounds it: reading K and V once.  In a tile of 128 rows the tensor-core
// forward fills one to eight, and its chain of products and exponentials takes
// 1 us a tile of keys; binary32 would first write its pieces.  Here the FMA pipe
// does it: a key's row lies in L lanes, 16 bytes each, which hold the same
// channels of all query rows in registers; a dot product takes log2(L)
// shuffles.  Each group of L lanes walks its own keys (32 / L a warp at once, U
// times that loaded a step ahead) with its own running maximum and sum; groups,
// warps and, through the workspace, blocks are joined in a fixed order.  8 x
// 22223 keys of 8 heads of 64, one row: bf16 5.6 TB/s, binary32 6.1 TB/s.  Four
// rows (binary32, 2 heads) reach 3.1 TB/s: a dot product takes log2(L) shuffles a
// row, and four blocks an SM leave 128 registers, of which four rows spill up to
// 80 bytes and eight up to 268.
#include "msda_attention.cuh"
#include "msda_attention_decode.cuh"

namespace msda {

namespace {

constexpr int kDecodeWarps = 4;

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static __device__ __forceinline__ void get(const uint4& x, float (&v)[4]) {
        v[0] = __uint_as_float(x.x), v[1] = __uint_as_float(x.y), v[2] = __uint_as_float(x.z), v[3] = __uint_as_float(x.w);
    }
    static __device__ __forceinline__ float round(float x) { return x; }
};
template <>
struct Vec<__nv_bfloat16> {
    static __device__ __forceinline__ void get(const uint4& x, float (&v)[8]) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    static __device__ __forceinline__ __nv_bfloat16 round(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Vec<__half> {
    static __device__ __forceinline__ void get(const uint4& x, float (&v)[8]) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ __half round(float x) { return __float2half_rn(x); }
};

__device__ __forceinline__ float decode_ex2(float x) {  // 2 units in the last place; 0 for -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// joins (m2, l2, o2) to (m, l, o)
template <int E>
__device__ __forceinline__ void join(float& m, float& l, float (&o)[E], float m2, float l2, const float (&o2)[E]) {
    const float top = fmaxf(m, m2);
    const float f = m == -attn_inf() ? 0.f : exp2f(m - top), f2 = m2 == -attn_inf() ? 0.f : exp2f(m2 - top);
    m = top, l = l * f + l2 * f2;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + o2[e] * f2;
}

}  // namespace

// L: lanes a key; R: query rows held (row r: query r / G, head n G + r % G)
template <typename T, int L, int R>
__global__ void __launch_bounds__(kDecodeWarps * 32, 4) msda_attention_decode_kernel(const AttentionArgs a) {
    constexpr int E = 16 / (int)sizeof(T), K = 32 / L, U = R > 4 ? 2 : 4;
    __shared__ float part[kDecodeWarps][R][L * E + 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % L, group = lane / L;
    long long id = blockIdx.x;
    const int split = (int)(id % a.splits);
    id /= a.splits;
    const int n = (int)(id % a.N), b = (int)(id / a.N), rows = a.Q * a.G;
    const bool in = c * E < a.D;  // D is a multiple of E
    const T* key = static_cast<const T*>(a.k) + b * a.k_sb + n * a.k_sh + c * E;
    const T* value = static_cast<const T*>(a.v) + b * a.v_sb + n * a.v_sh + c * E;
    const uint8_t* km = a.key_mask ? a.key_mask + b * a.km_sb : nullptr;
    float q[R][E], o[R][E], m[R], l[R];
    const uint8_t* mask[R];
    int seen[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int qi = r / a.G, h = n * a.G + r % a.G;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < rows && in) x = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + b * a.q_sb + qi * a.q_ss + h * a.q_sh + c * E);
        Vec<T>::get(x, q[r]);
        mask[r] = a.mask ? a.mask + b * a.mk_sb + h * a.mk_sh + qi * a.mk_sq : nullptr;
        seen[r] = r >= rows ? 0 : a.causal ? min(a.S, max(0, qi + 1 + (a.S - a.Q))) : a.S;
        m[r] = -attn_inf(), l[r] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[r][e] = 0.f;
    }
    const int j0 = split * a.tiles_per_split, j1 = min(a.S, j0 + a.tiles_per_split);
    uint32_t ahead[U];  // a bit a row
    uint4 kn[U], vn[U];
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = base + u * K + group;
            ahead[u] = 0;
            if (j < j1 && (!km || km[j])) {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (j < seen[r] && (!a.mask || mask[r][j])) ahead[u] |= 1u << r;
            }
            kn[u] = vn[u] = make_uint4(0, 0, 0, 0);
            if (ahead[u] && in) {
                kn[u] = *reinterpret_cast<const uint4*>(key + j * a.k_ss);
                vn[u] = *reinterpret_cast<const uint4*>(value + j * a.v_ss);
            }
        }
    };
    const int step = kDecodeWarps * K * U;
    load(j0 + warp * K * U);
    for (int base = j0 + warp * K * U; base < j1; base += step) {
        uint32_t on[U];
        uint4 kx[U], vx[U];
#pragma unroll
        for (int u = 0; u < U; ++u) on[u] = ahead[u], kx[u] = kn[u], vx[u] = vn[u];
        load(base + step);
        float s[U][R];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[E];
            Vec<T>::get(kx[u], x);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float d = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) d = fmaf(q[r][e], x[e], d);
#pragma unroll
                for (int w = L / 2; w > 0; w >>= 1) d += __shfl_xor_sync(0xffffffffu, d, w);
                s[u][r] = (on[u] >> r) & 1u ? d * a.c2 : -attn_inf();
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float top = m[r];
#pragma unroll
            for (int u = 0; u < U; ++u) top = fmaxf(top, s[u][r]);
            const float ref = top == -attn_inf() ? 0.f : top, f = decode_ex2(m[r] - ref);
            m[r] = top, l[r] *= f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[r][e] *= f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[u][r] = decode_ex2(s[u][r] - ref);
                l[r] += s[u][r];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[E];
            Vec<T>::get(vx[u], x);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int e = 0; e < E; ++e) o[r][e] = fmaf(s[u][r], x[e], o[r][e]);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int w = L; w < 32; w <<= 1) {
            float o2[E];
#pragma unroll
            for (int e = 0; e < E; ++e) o2[e] = __shfl_xor_sync(0xffffffffu, o[r][e], w);
            join<E>(m[r], l[r], o[r], __shfl_xor_sync(0xffffffffu, m[r], w), __shfl_xor_sync(0xffffffffu, l[r], w), o2);
        }
        if (group == 0) {
#pragma unroll
            for (int e = 0; e < E; ++e) part[warp][r][2 + c * E + e] = o[r][e];
            if (c == 0) part[warp][r][0] = m[r], part[warp][r][1] = l[r];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * L * E; i += kDecodeWarps * 32) {
        const int r = i / (L * E), d = i - r * (L * E);
        float top = -attn_inf();
#pragma unroll
        for (int w = 0; w < kDecodeWarps; ++w) top = fmaxf(top, part[w][r][0]);
        float sum = 0.f, x = 0.f;
#pragma unroll
        for (int w = 0; w < kDecodeWarps; ++w) {
            const float f = top == -attn_inf() ? 1.f : exp2f(part[w][r][0] - top);  // none seen: zeros, or NaN scores alone
            sum += part[w][r][1] * f;
            x += part[w][r][2 + d] * f;
        }
        const float l2 = sum == 0.f ? -attn_inf() : top + log2f(sum);
        x = sum == 0.f ? 0.f : x / sum;
        const int qi = r / a.G, h = n * a.G + r % a.G;
        const long long row = ((long long)b * a.M + h) * a.Q + qi, at = (long long)split * a.B * a.M * a.Q + row;
        if (a.splits > 1) {
            if (d < a.D) a.part_o[at * a.D + d] = x;
            if (d == 0) a.part_lse[at] = l2;
        } else {
            if (d < a.D) static_cast<T*>(a.out)[(((long long)b * a.Q + qi) * a.M + h) * a.D + d] = Vec<T>::round(x);
            if (d == 0) a.lse[row] = l2 * kLn2;
        }
    }
}

template <typename T, int L>
static cudaError_t decode_rows(const AttentionArgs& a, unsigned grid, cudaStream_t st) {
    const int rows = a.Q * a.G;
    if (rows == 1) {
        msda_attention_decode_kernel<T, L, 1><<<grid, kDecodeWarps * 32, 0, st>>>(a);
    } else if constexpr (sizeof(T) == 4) {
        if (rows <= 4) msda_attention_decode_kernel<T, L, 4><<<grid, kDecodeWarps * 32, 0, st>>>(a);
        else msda_attention_decode_kernel<T, L, 8><<<grid, kDecodeWarps * 32, 0, st>>>(a);
    }
    return cudaGetLastError();
}
template <typename T>
cudaError_t launch_attention_decode(const AttentionArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)((long long)a.B * a.N * a.splits);
    const int lanes = a.D * (int)sizeof(T) / 16;
    if (lanes <= 4) return decode_rows<T, 4>(a, grid, st);
    if (lanes <= 8) return decode_rows<T, 8>(a, grid, st);
    if (lanes <= 16) return decode_rows<T, 16>(a, grid, st);
    if constexpr (sizeof(T) == 4) return decode_rows<T, 32>(a, grid, st);
    return cudaErrorInvalidValue;  // 16-bit rows have 16 vectors at most
}
template cudaError_t launch_attention_decode<float>(const AttentionArgs&, cudaStream_t);
template cudaError_t launch_attention_decode<__half>(const AttentionArgs&, cudaStream_t);
template cudaError_t launch_attention_decode<__nv_bfloat16>(const AttentionArgs&, cudaStream_t);

}  // namespace msda
