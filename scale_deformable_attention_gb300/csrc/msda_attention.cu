// msda_attention.cu -- host side of msda_attention_forward / _backward:
// checks, workspace layout, choice of kernels, launches.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <limits>

#include "msda_attention.cuh"
#include "msda_attention_decode.cuh"
#include "msda_attention_simt.cuh"
#include "msda_attention_tc_host.cuh"
#include "msda_host.cuh"

namespace msda {

// One pass over a mask of bytes [Bm, Mm, Q, S]; with `causal` a pair that it hides
// counts as masked.  Writes
//   live [LB, LN, S] bytes (cleared before): 1 where some query of the heads that
//     share the key sees it; a key outside it may hold anything, NaN too (every
//     writer of a byte writes the same 1);
//   bits [Bm, Mm, Q, W] and bits_t [Bm, Mm, S, Wq] (tensor-core kernels; or
//     null): the mask and its transpose, 32 pairs a word, zeros behind S and Q;
//   ext_q, ext_k (cleared before): where a tile of queries, and one of keys, begins and ends (see TcArgs; maxima of
//     integers, the same in any order).
// A warp takes 32 queries and 128 keys, a lane four keys: one 32-bit load a row
// where the row's address allows it, else four of a byte.  A row's words are
// put together by eight lanes each, the keys' columns build up in each lane.
// (One key a lane took 330 us for 16000 x 16000 pairs, four times the loads.)
__global__ void __launch_bounds__(128) msda_attention_mask_kernel(const uint8_t* mask, long long mk_sb, long long mk_sh,
                                                                  long long mk_sq, const uint8_t* key_mask,
                                                                  long long km_sb, int Q, int S, int G, int Bm, int Mm,
                                                                  int LB, int LN, int B, int causal, uint8_t* live, uint32_t* bits,
                                                                  uint32_t* bits_t, int W, int Wq, int2* ext_q, int2* ext_k) {
    const int lane = threadIdx.x & 31, j = blockIdx.x * 128 + lane * 4, n = S - j < 4 ? S - j : 4;  // the lane's keys: n > 0 of them
    for (int z = blockIdx.z; z < Bm * Mm; z += gridDim.z) {
        const int bm = z / Mm, mm = z - bm * Mm;
        const uint8_t* src = mask + bm * mk_sb + mm * mk_sh + j;
        for (int qt = blockIdx.y; qt < Wq / 4; qt += gridDim.y) {
            const int qw = qt * 4 + (threadIdx.x >> 5), q0 = qw * 32;
            uint32_t row[4] = {}, col[4] = {};
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += 16) {
                uint32_t v[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const uint8_t* at = src + (q0 + r0 + r) * mk_sq;
                    v[r] = 0;
                    if (q0 + r0 + r < Q) {
                        if (n == 4 && (reinterpret_cast<uintptr_t>(at) & 3) == 0) {
                            v[r] = *reinterpret_cast<const uint32_t*>(at);
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (e < n) v[r] |= (uint32_t)at[e] << (8 * e);
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    uint32_t four = ((__vcmpne4(v[r], 0u) & 0x08040201u) * 0x01010101u) >> 24;  // a bit a key
                    if (causal) four &= tc_low_bits(q0 + r0 + r + (S - Q) - j + 1);
                    uint32_t w = four << (4 * (lane & 7));
                    w |= __shfl_xor_sync(0xffffffffu, w, 1);
                    w |= __shfl_xor_sync(0xffffffffu, w, 2);
                    w |= __shfl_xor_sync(0xffffffffu, w, 4);
                    if ((lane & 7) == (r & 7)) row[(r0 + r) >> 3] = w;
#pragma unroll
                    for (int e = 0; e < 4; ++e) col[e] |= ((four >> e) & 1u) << (r0 + r);
                }
            }
            if (bits) {
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int q = q0 + t * 8 + (lane & 7);
                    if (q < Q) bits[((long long)z * Q + q) * W + blockIdx.x * 4 + (lane >> 3)] = row[t];
                }
            }
            if (bits_t) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < n) bits_t[((long long)z * S + j + e) * Wq + qw] = col[e];
            }
            const uint32_t any = col[0] | col[1] | col[2] | col[3];
            if (__any_sync(0xffffffffu, any != 0) && lane < 4) {
                int2* e = lane < 2 ? ext_q + (long long)z * (Wq / 4) + qt : ext_k + (long long)z * (W / 4) + blockIdx.x;
                const int t = lane < 2 ? (int)blockIdx.x : qt, v = lane & 1 ? t + 1 : kTcFar - t;
                atomicMax(lane & 1 ? &e->y : &e->x, v);
            }
            if (any) {
                const int ln = LN > 1 ? mm / G : 0;
                // a mask that all batch items share meets the key_mask of each
                const int b0 = Bm > 1 ? bm : 0, b1 = Bm > 1 ? bm + 1 : LB;
                for (int b = b0; b < b1; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (col[e] && (!key_mask || key_mask[b * km_sb + j + e]))
                            live[((long long)(LB > 1 ? b : 0) * LN + ln) * S + j + e] = 1;
            }
        }
    }
}

}  // namespace msda

namespace {

using msda::AttentionArgs;
using msda::AttentionRows;
using msda::failf;
using msda::kPlanSms;

constexpr unsigned kFlags = MSDA_ATTENTION_CAUSAL | MSDA_ATTENTION_KEY_MASK | MSDA_ATTENTION_MASK;

size_t up(size_t n) { return (n + 255) / 256 * 256; }

// Tensors that the tensor-core kernels take where their addresses and strides
// are made of 16 bytes: 16-bit, channels in whole 16-byte vectors, a group of
// shared heads that fits a tile, some key.
bool tc_type(msda_dtype dt, const msda_attention_problem* p) {
    return dt != MSDA_F32 && p->D % 8 == 0 && p->M / p->N <= 128 && p->S > 0;
}

// binary32 that the tensor cores take in three bf16 pieces, whatever its
// addresses and strides: up to 64 channels (an operand's pieces of a tile take
// 48 KB), and enough pairs to pay for the cutting.  Against the FMA pipe, all
// launches in one graph, 8 heads: forward 22 : 15 us at 300 x 300 and 27 : 17 at 900 x 900 of one
// head, 25 : 34 at four times 300 x 300, 35 : 49 at 64 x 4000 and 45 : 128 at 1 x 20000 (FMA-pipe blocks take 64 rows, which
// the count rounds up to; 64 keys fill half a tile: 45 : 21 at 64 times 64 x 64).  Backward: 59 : 81 us at 64 times 64 x 64
// against 31 : 38 at 100 x 100, 49 : 81 at 300 x 300, 202 : 901 at 4000 x 64.
bool tc_pieces(msda_dtype dt, const msda_attention_problem* p, bool backward) {
    if (dt != MSDA_F32 || p->D > 64 || p->M / p->N > 128 || p->S == 0) return false;
    if (backward) return p->Q > 64 || p->S > 64;
    return p->S > 64 && p->B * p->M * ((p->Q + 63) / 64) * ((p->S + 63) / 64) >= 3 << 7;  // tiles of 64 x 64
}

// A few rows over many keys, where addresses and strides are made of 16 bytes: one row in 16 bits, up to eight in
// binary32.  In 16 bits (8 x 22223 keys of 8 heads of 64: 65 us against 78 on the tensor cores; 64 x 300 of 8 of 128: 13
// against 30) more rows cost this form in proportion and a tile of the tensor cores nothing (four rows, 8 x 22223 of 2
// of 64: 45 against 26).  binary32: one row 120 against 567, four 58 against 162, eight (1 x 22223 of 8 of 64) 58 against 94.
bool decode_shape(msda_dtype dt, const msda_attention_problem* p) {
    const int64_t rows = p->Q * (p->M / p->N);
    return p->S >= 256 && (dt == MSDA_F32 ? rows <= msda::kDecodeRows && p->D % 4 == 0 : rows == 1 && p->D % 8 == 0);
}
// Keys a block of four warps takes, 128 at least: one wave of the four blocks that an SM holds (at 4.2 an SM 94 us, not 66).
void decode_splits(const msda_attention_problem* p, int* splits, int* per) {
    const int64_t heads = p->B * p->N, most = (p->S + 127) / 128;
    int64_t n = heads > 0 ? 4 * kPlanSms / heads : 1;
    if (n < 1) n = 1;
    if (n > most) n = most;
    const int64_t each = (p->S + n - 1) / n;
    *per = (int)each;
    *splits = (int)((p->S + each - 1) / each);
}

// The pieces in the workspace: the flag, then query, key, value and (backward) the output's gradient.
struct PieceSpace {
    int Dp;
    size_t q, k, v, g, bytes;
};
PieceSpace piece_space(const msda_attention_problem* p, bool backward) {
    PieceSpace s;
    s.Dp = (int)((p->D + 7) / 8 * 8);
    const size_t rows = up((size_t)p->B * p->Q * p->M * s.Dp * 6), keys = up((size_t)p->B * p->S * p->N * s.Dp * 6);
    s.q = 256, s.k = s.q + rows, s.v = s.k + keys, s.g = s.v + keys;
    s.bytes = s.g + (backward ? rows : 0);
    return s;
}

msda_status check(msda_dtype dt, unsigned flags, const msda_attention_problem* p) {
    if (dt != MSDA_F32 && dt != MSDA_F16 && dt != MSDA_BF16) return failf(MSDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
    if (flags & ~kFlags) return failf(MSDA_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    if (!p) return failf(MSDA_ERR_INVALID_ARG, "problem is NULL");
    if (p->B < 0 || p->Q < 0 || p->S < 0) return failf(MSDA_ERR_INVALID_ARG, "negative size (B=%lld Q=%lld S=%lld)",
                                                      (long long)p->B, (long long)p->Q, (long long)p->S);
    if (p->M < 1 || p->N < 1 || p->D < 1)
        return failf(MSDA_ERR_INVALID_ARG, "M=%lld, N=%lld and D=%lld must be at least 1", (long long)p->M,
                     (long long)p->N, (long long)p->D);
    if (p->M % p->N) return failf(MSDA_ERR_INVALID_ARG, "N=%lld key heads do not divide M=%lld query heads",
                                  (long long)p->N, (long long)p->M);
    if (p->D > msda::kAttnMaxChannels)
        return failf(MSDA_ERR_UNSUPPORTED, "D=%lld above %d", (long long)p->D, msda::kAttnMaxChannels);
    const int64_t top = 1ll << 30;
    if (p->Q > top || p->S > top || p->M > 65535 || p->B > top)
        return failf(MSDA_ERR_UNSUPPORTED, "B=%lld, Q=%lld, S=%lld or M=%lld too large", (long long)p->B, (long long)p->Q,
                     (long long)p->S, (long long)p->M);
    int64_t t;
    if (!msda::mul_fits(p->B, p->M, &t) || !msda::mul_fits(t, (p->Q > p->S ? p->Q : p->S) + 256, &t) ||
        !msda::mul_fits(t, p->D * 512, &t))
        return failf(MSDA_ERR_INVALID_ARG, "B*M*max(Q,S)*D overflows 64 bits");
    // one block takes 64 or 128 rows of a head
    if (p->B * p->M * ((p->Q + 63) / 64) > 0x7fffffffll || p->B * p->N * ((p->S + 63) / 64) > 0x7fffffffll || p->B * p->N > 0x3fffffffll)
        return failf(MSDA_ERR_UNSUPPORTED, "more than 2^31 - 1 blocks of rows");
    const int64_t* st[] = {p->query_stride, p->key_stride, p->value_stride, p->mask_stride};
    for (const int64_t* s : st)
        for (int i = 0; i < 3; ++i)
            if (s[i] < 0) return failf(MSDA_ERR_INVALID_ARG, "negative stride");
    if (p->key_mask_stride < 0) return failf(MSDA_ERR_INVALID_ARG, "negative stride");
    return MSDA_OK;
}

// What the mask becomes in the workspace: the liveness of keys [LB][LN][S]
// bytes, the pairs as bits by query and, for the tensor-core kernels, by key.
struct MaskSpace {
    int Bm = 1, Mm = 1, LB = 1, LN = 1, W = 0, Wq = 0;
    size_t ext_q = 0, ext_k = 0, bits = 0, bits_t = 0, bytes = 0;  // offsets behind the liveness; what lies before `bits` is cleared
};
MaskSpace mask_space(unsigned flags, const msda_attention_problem* p, bool by_key) {
    MaskSpace l;
    if (!(flags & MSDA_ATTENTION_MASK)) return l;
    l.Bm = p->B > 1 && p->mask_stride[0] != 0 ? (int)p->B : 1;
    l.Mm = p->M > 1 && p->mask_stride[1] != 0 ? (int)p->M : 1;
    l.LB = (flags & MSDA_ATTENTION_KEY_MASK) || l.Bm > 1 ? (int)p->B : 1;
    l.LN = l.Mm > 1 ? (int)p->N : 1;
    l.W = (int)((p->S + 127) / 128 * 4);
    l.Wq = (int)((p->Q + 127) / 128 * 4);
    l.ext_q = up((size_t)l.LB * l.LN * (size_t)p->S);
    l.ext_k = l.ext_q + (size_t)l.Bm * l.Mm * (l.Wq / 4) * 8;
    l.bits = up(l.ext_k + (size_t)l.Bm * l.Mm * (l.W / 4) * 8);
    l.bits_t = l.bits + up((size_t)l.Bm * l.Mm * p->Q * l.W * 4);
    l.bytes = l.bits_t;
    if (by_key) l.bytes += up((size_t)l.Bm * l.Mm * p->S * l.Wq * 4);
    return l;
}

struct ForwardPlan {
    int G, qpt, nq, qblocks, splits, per;  // heads and queries a row tile, row tiles a block, blocks, split of the key axis
};

// Split of the key axis of the FMA-pipe forward: enough blocks for four a SM,
// so that a single query over a long key axis uses the whole GPU.
// 16-bit tensors that come here for their addresses alone split no further than
// the tensor-core form would, so that the workspace is that form's.
ForwardPlan forward_plan(const msda_attention_problem* p, int most_tiles = 2);
void simt_splits(msda_dtype dt, const msda_attention_problem* p, int* splits, int* per) {
    const int64_t blocks = p->B * p->M * ((p->Q + 63) / 64), tiles = (p->S + 63) / 64;
    int64_t n = 1;
    if (blocks > 0 && blocks < 2 * kPlanSms && tiles > 1) {
        n = (4 * kPlanSms + blocks - 1) / blocks;
        if (n > tiles) n = tiles;
        if (n > 64) n = 64;
        if (tc_type(dt, p)) {
            const int64_t most = forward_plan(p).splits;
            if (n > most) n = most;
        }
    }
    const int64_t each = tiles > 0 ? (tiles + n - 1) / n : 1;
    *per = (int)each;
    *splits = tiles > 0 ? (int)((tiles + each - 1) / each) : 1;
}

size_t part_bytes(const msda_attention_problem* p, int splits) {
    if (splits <= 1) return 0;
    const size_t rows = (size_t)splits * p->B * p->M * p->Q;
    return up(rows * p->D * 4) + up(rows * 4);
}

msda_status masks_ok(unsigned flags, const msda_attention_problem* p, const uint8_t* key_mask, const uint8_t* mask) {
    const bool any = p->B > 0 && p->S > 0;
    const struct { unsigned bit; const void* p; bool need; const char* name; } m[] = {
        {MSDA_ATTENTION_KEY_MASK, key_mask, any, "key_mask"}, {MSDA_ATTENTION_MASK, mask, any && p->Q > 0, "mask"}};
    for (const auto& x : m) {
        if ((flags & x.bit) && x.need && !x.p) return failf(MSDA_ERR_INVALID_ARG, "%s is NULL", x.name);
        if (!(flags & x.bit) && x.p) return failf(MSDA_ERR_INVALID_ARG, "%s is given without its flag", x.name);
    }
    return MSDA_OK;
}

AttentionArgs args_of(unsigned flags, const msda_attention_problem* p, double scale, const void* q, const void* k,
                      const void* v, const uint8_t* key_mask, const uint8_t* mask) {
    AttentionArgs a{};
    a.q = q, a.k = k, a.v = v;
    a.q_sb = p->query_stride[0], a.q_ss = p->query_stride[1], a.q_sh = p->query_stride[2];
    a.k_sb = p->key_stride[0], a.k_ss = p->key_stride[1], a.k_sh = p->key_stride[2];
    a.v_sb = p->value_stride[0], a.v_ss = p->value_stride[1], a.v_sh = p->value_stride[2];
    a.key_mask = key_mask, a.km_sb = p->key_mask_stride;
    a.mask = mask, a.mk_sb = p->mask_stride[0], a.mk_sh = p->mask_stride[1], a.mk_sq = p->mask_stride[2];
    a.B = (int)p->B, a.Q = (int)p->Q, a.S = (int)p->S, a.M = (int)p->M, a.N = (int)p->N, a.D = (int)p->D;
    a.G = (int)(p->M / p->N);
    a.causal = (flags & MSDA_ATTENTION_CAUSAL) != 0;
    a.scale = (float)scale;
    // never 0, by which the -inf of a masked pair would become NaN (a score is then off by 2^-149 |q k|, below 2^-20)
    a.c2 = std::fmax((float)(scale * 1.4426950408889634), std::numeric_limits<float>::denorm_min());
    a.splits = 1;
    a.tiles_per_split = 1 << 30;
    return a;
}

// Replaces key_mask by the keys that some pair of the mask leaves, and brings
// the mask's bits up (by key where asked for).
msda_status make_mask(AttentionArgs& a, const MaskSpace& l, void* ws, msda::TcArgs& t, bool by_key, cudaStream_t st) {
    if (!a.mask) return MSDA_OK;
    uint8_t* live = static_cast<uint8_t*>(ws);
    uint32_t* bits = reinterpret_cast<uint32_t*>(live + l.bits);
    int2 *ext_q = reinterpret_cast<int2*>(live + l.ext_q), *ext_k = reinterpret_cast<int2*>(live + l.ext_k);
    uint32_t* bits_t = by_key ? reinterpret_cast<uint32_t*>(live + l.bits_t) : nullptr;
    if (a.S > 0) {
        msda::TraceSpan ts(st);
        cudaError_t e = cudaMemsetAsync(live, 0, l.bits, st);
        if (e == cudaSuccess) {
            const int64_t z = (int64_t)l.Bm * l.Mm;
            const dim3 grid((unsigned)((a.S + 127) / 128), (unsigned)(l.Wq / 4 < 65535 ? l.Wq / 4 : 65535),
                            (unsigned)(z < 65535 ? z : 65535));
            msda::msda_attention_mask_kernel<<<grid, 128, 0, st>>>(a.mask, a.mk_sb, a.mk_sh, a.mk_sq, a.key_mask, a.km_sb, a.Q,
                                                                   a.S, a.G, l.Bm, l.Mm, l.LB, l.LN, a.B, a.causal, live, bits, bits_t,
                                                                   l.W, l.Wq, ext_q, ext_k);
            e = cudaGetLastError();
        }
        ts.end(MSDA_KERNEL_ATTENTION_MASK, (int64_t)a.Q * a.S);
        if (e != cudaSuccess) return failf(MSDA_ERR_CUDA, "mask kernel launch: %s", cudaGetErrorString(e));
    }
    a.key_mask = live;
    a.km_sb = l.LB > 1 ? (long long)l.LN * a.S : 0;
    a.km_sh = l.LN > 1 ? a.S : 0;
    a.bits = bits, a.W = l.W;
    a.bits_sh = l.Mm > 1 ? (long long)a.Q * l.W : 0;
    a.bits_sb = l.Bm > 1 ? (long long)l.Mm * a.Q * l.W : 0;
    t.ext_q = ext_q, t.ext_k = ext_k;
    t.ext_sh = l.Mm > 1 ? 1 : 0, t.ext_sb = l.Bm > 1 ? l.Mm : 0;
    t.bits_t = bits_t, t.Wq = l.Wq;
    t.bits_t_sh = l.Mm > 1 ? (long long)a.S * l.Wq : 0;
    t.bits_t_sb = l.Bm > 1 ? (long long)l.Mm * a.S * l.Wq : 0;
    return MSDA_OK;
}

using EncodeTiled = PFN_cuTensorMapEncodeTiled_v12000;

// Rows of a [B, rows, heads, D] tensor as (channel, head of the group, row,
// key head, batch); boxes of 64 channels x G heads x `rows` rows with the
// 128-byte swizzle; zeros outside.
bool rows_map(msda_dtype dt, const void* base, int64_t D, int64_t G, int64_t rows, int64_t N, int64_t B, int64_t sb,
              int64_t ss, int64_t sh, int box_rows, CUtensorMap* map) {
    EncodeTiled f = reinterpret_cast<EncodeTiled>(msda::tensor_map_encoder());
    if (!f) return false;
    // the stride of a dimension of one element is never used, and need not be a whole number of vectors
    auto bytes = [](int64_t n, int64_t stride) { return (cuuint64_t)(n > 1 ? stride * 2 : 16); };
    const cuuint64_t dims[5] = {(cuuint64_t)D, (cuuint64_t)G, (cuuint64_t)rows, (cuuint64_t)N, (cuuint64_t)B};
    const cuuint64_t strides[4] = {bytes(G, sh), bytes(rows, ss), bytes(N, G * sh), bytes(B, sb)};
    const cuuint32_t box[5] = {64u, (cuuint32_t)G, (cuuint32_t)box_rows, 1u, 1u};
    const cuuint32_t one[5] = {1u, 1u, 1u, 1u, 1u};
    return f(map, dt == MSDA_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
             const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether TMA can read a tensor: 16-byte address, strides of whole vectors below 2^40 bytes.
bool tma_rows(const void* p, const int64_t* stride, int64_t B, int64_t rows, int64_t heads) {
    const int64_t n[3] = {B, rows, heads};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (stride[i] % 8 || stride[i] <= 0 || stride[i] >= (1ll << 38) / heads)) return false;
    return msda::aligned_to(p, 16);
}

// Whether rows are made of 16-byte vectors of `v` elements.
bool vector_rows(const void* x, const int64_t* stride, int64_t v, int64_t B, int64_t rows, int64_t heads) {
    const int64_t n[3] = {B, rows, heads};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && stride[i] % v) return false;
    return msda::aligned_to(x, 16);
}

// Row blocks and split of the tensor-core forward.  Two row tiles a block
// overlap one's products with the other's exponentials; one tile where two
// would leave SMs without a block, or where the last round of blocks eats the gain.  A key axis of many tiles is split until
// every SM has a block, but not into pieces of less than four tiles: a piece
// costs a launch's start and the joining of its rows.
ForwardPlan forward_plan(const msda_attention_problem* p, int most_tiles) {
    ForwardPlan f;
    f.G = (int)(p->M / p->N);
    f.qpt = msda::kTcRows / f.G;
    const int64_t one = (p->Q + f.qpt - 1) / f.qpt, two = (p->Q + 2 * f.qpt - 1) / (2 * f.qpt);
    // rounds of blocks, one an SM; a step of two tiles takes about three halves of a step of one
    const int64_t heads = p->B * p->N, rounds1 = (heads * one + kPlanSms - 1) / kPlanSms, rounds2 = (heads * two + kPlanSms - 1) / kPlanSms;
    f.nq = most_tiles == 2 && heads * two >= kPlanSms && 3 * rounds2 <= 2 * rounds1 ? 2 : 1;
    f.qblocks = (int)(f.nq == 2 ? two : one);
    const int64_t blocks = p->B * p->N * f.qblocks, tiles = (p->S + msda::kTcRows - 1) / msda::kTcRows;
    int64_t n = blocks > 0 ? kPlanSms / blocks : 1;
    if (n > tiles / 4) n = tiles / 4;
    if (n < 1) n = 1;
    const int64_t each = tiles > 0 ? (tiles + n - 1) / n : 1;
    f.per = (int)each;
    f.splits = tiles > 0 ? (int)((tiles + each - 1) / each) : 1;
    return f;
}

bool simt_vec(const AttentionArgs& a) {  // binary32 rows read as 16-byte vectors
    const long long st[] = {a.q_sb, a.q_ss, a.q_sh, a.k_sb, a.k_ss, a.k_sh, a.v_sb, a.v_ss, a.v_sh, a.D};
    for (long long s : st)
        if (s % 4) return false;
    return msda::aligned_to(a.q, 16) && msda::aligned_to(a.k, 16) && msda::aligned_to(a.v, 16) &&
           msda::aligned_to(a.dout, 16);
}

// A tensor's three pieces: boxes of `box_rows` rows of `group` heads.
bool piece_map(const msda_attention_problem* p, const void* base, int group, int64_t rows, int64_t heads, int box_rows,
               CUtensorMap* map) {
    const int64_t Dp = (p->D + 7) / 8 * 8, row = heads * group * Dp;
    return rows_map(MSDA_BF16, base, Dp, group, rows, heads, 3 * p->B, rows * row, row, Dp, box_rows, map);
}

#define MSDA_BY_DTYPE(dt, f, ...)                       \
    ((dt) == MSDA_F32   ? msda::f<float>(__VA_ARGS__)   \
     : (dt) == MSDA_F16 ? msda::f<__half>(__VA_ARGS__)  \
                        : msda::f<__nv_bfloat16>(__VA_ARGS__))

msda_status launched(cudaError_t e, const char* what) {
    return e == cudaSuccess ? MSDA_OK : failf(MSDA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

msda_status join_parts(msda_dtype dt, const AttentionArgs& a, const msda_attention_problem* p, cudaStream_t st) {
    msda::TraceSpan ts(st);
    const msda_status s = launched(MSDA_BY_DTYPE(dt, launch_attention_join, a, st), "attention join kernel launch");
    ts.end(MSDA_KERNEL_ATTENTION_JOIN, p->B * p->M * p->Q);
    return s;
}

// Clears the flag and cuts the tensors; a.key_mask (and, backward, lse) say which rows take part.
msda_status make_pieces(AttentionArgs& a, const msda_attention_problem* p, const float* lse, unsigned char* ws, cudaStream_t st) {
    const PieceSpace w = piece_space(p, a.dout != nullptr);
    unsigned* odd = reinterpret_cast<unsigned*>(ws);
    msda::SplitArgs s{};
    const bool vec = simt_vec(a);
    auto f = [](const void* x) { return static_cast<const float*>(x); };
    s.t[0] = {f(a.q), a.q_sb, a.q_ss, a.q_sh, a.Q, a.M, vec, nullptr, 0, 0, lse, ws + w.q};
    s.t[1] = {f(a.k), a.k_sb, a.k_ss, a.k_sh, a.S, a.N, vec, a.key_mask, a.km_sb, a.km_sh, nullptr, ws + w.k};
    s.t[2] = {f(a.v), a.v_sb, a.v_ss, a.v_sh, a.S, a.N, vec, a.key_mask, a.km_sb, a.km_sh, nullptr, ws + w.v};
    s.t[3] = {f(a.dout), (long long)a.Q * a.M * a.D, (long long)a.M * a.D, a.D, a.Q, a.M, vec, nullptr, 0, 0, lse, ws + w.g};
    s.B = a.B, s.D = a.D, s.Dp = w.Dp, s.odd = odd;
    a.odd = odd;
    msda::TraceSpan ts(st);
    cudaError_t e = cudaMemsetAsync(odd, 0, 4, st);
    if (e == cudaSuccess) e = msda::launch_attention_split(s, a.dout ? 4 : 3, st);
    ts.end(MSDA_KERNEL_ATTENTION_SPLIT, p->B * p->M * p->Q);
    return launched(e, "attention split kernel launch");
}

// Workspace of the backward: the rows' statistics, f16's norms, the mask.
// Row tiles are 128 rows on the tensor cores, 64 on the FMA pipe; which runs
// depends on the addresses, and 128 needs as much space or more.
struct BackwardLayout {
    AttentionRows rows;
    size_t l2 = 0, top = 0, mask = 0, pieces = 0, bytes = 0;
};
BackwardLayout backward_layout(msda_dtype dt, unsigned flags, const msda_attention_problem* p, bool tc) {
    BackwardLayout w;
    const int rt = tc ? msda::kTcRows : 64;
    w.rows = {rt, (int)((p->Q + rt - 1) / rt), (int)p->M};
    const size_t n = up((size_t)p->B * w.rows.heads * w.rows.tiles * w.rows.rt * 8);
    w.top = n;
    w.mask = n + 256;
    w.pieces = w.mask + mask_space(flags, p, tc_type(dt, p) || tc_pieces(dt, p, true)).bytes;
    w.bytes = w.pieces + (tc_pieces(dt, p, true) ? piece_space(p, true).bytes : 0);
    return w;
}

}  // namespace

extern "C" {

size_t msda_attention_forward_workspace_size(msda_dtype dt, unsigned flags, const msda_attention_problem* p) {
    if (check(dt, flags, p) != MSDA_OK) return 0;
    int splits, per;
    simt_splits(dt, p, &splits, &per);
    if (tc_type(dt, p)) splits = forward_plan(p).splits;  // which of the two runs depends on the addresses
    size_t pieces = 0;
    if (tc_pieces(dt, p, false)) splits = forward_plan(p, 1).splits, pieces = piece_space(p, false).bytes;
    size_t need = part_bytes(p, splits) + mask_space(flags, p, false).bytes + pieces;
    if (decode_shape(dt, p)) {
        decode_splits(p, &splits, &per);
        const size_t n = part_bytes(p, splits);
        if (n > need) need = n;
    }
    return need;
}

size_t msda_attention_backward_workspace_size(msda_dtype dt, unsigned flags, const msda_attention_problem* p) {
    if (check(dt, flags, p) != MSDA_OK) return 0;
    return backward_layout(dt, flags, p, tc_type(dt, p) || tc_pieces(dt, p, true)).bytes;
}

msda_status msda_attention_forward(msda_dtype dt, unsigned flags, const msda_attention_problem* p, double scale,
                                   const void* query, const void* key, const void* value, const uint8_t* key_mask,
                                   const uint8_t* mask, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                   msda_stream_t stream) {
    msda::clear_error();
    msda_status s = check(dt, flags, p);
    if (s != MSDA_OK) return s;
    if (!(scale > 0.0 && scale < 1e30)) return failf(MSDA_ERR_INVALID_ARG, "scale=%g must be positive", scale);
    const size_t es = dt == MSDA_F32 ? 4 : 2;
    const bool rows = p->B > 0 && p->Q > 0, keys = rows && p->S > 0;
    if ((s = msda::need_ptr(query, keys, es, "query")) || (s = msda::need_ptr(key, keys, es, "key")) ||
        (s = msda::need_ptr(value, keys, es, "value")) || (s = msda::need_ptr(out, rows, es, "out")) ||
        (s = msda::need_ptr(lse, rows, 4, "lse")) || (s = masks_ok(flags, p, key_mask, mask)))
        return s;
    if (!rows) return MSDA_OK;
    const size_t need = msda_attention_forward_workspace_size(dt, flags, p);
    if (need && (!workspace || workspace_bytes < need || !msda::aligned_to(workspace, 256)))
        return failf(MSDA_ERR_WORKSPACE, "workspace of %zu bytes, 256-byte aligned, needed (got %zu)", need, workspace_bytes);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    AttentionArgs a = args_of(flags, p, scale, query, key, value, key_mask, mask);
    a.out = out, a.lse = lse;
    const bool tc = tc_type(dt, p) && tma_rows(query, p->query_stride, p->B, p->Q, p->M) &&
                    tma_rows(key, p->key_stride, p->B, p->S, p->N) && tma_rows(value, p->value_stride, p->B, p->S, p->N) &&
                    msda::aligned_to(out, 16);
    const int64_t v = 16 / (int64_t)es;
    if (decode_shape(dt, p) && vector_rows(query, p->query_stride, v, p->B, p->Q, p->M) &&
        vector_rows(key, p->key_stride, v, p->B, p->S, p->N) && vector_rows(value, p->value_stride, v, p->B, p->S, p->N)) {
        decode_splits(p, &a.splits, &a.tiles_per_split);
        if (a.splits > 1) {
            a.part_o = static_cast<float*>(workspace);
            a.part_lse = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + up((size_t)a.splits * p->B * p->M * p->Q * p->D * 4));
        }
        {
            msda::TraceSpan ts(st);
            s = launched(MSDA_BY_DTYPE(dt, launch_attention_decode, a, st), "attention kernel launch");
            ts.end(MSDA_KERNEL_ATTENTION, p->B * p->M * p->Q);
        }
        return s == MSDA_OK && a.splits > 1 ? join_parts(dt, a, p, st) : s;
    }
    const MaskSpace ms = mask_space(flags, p, false);
    msda::TcArgs t{};
    const bool pieces = tc_pieces(dt, p, false);
    if ((s = make_mask(a, ms, workspace, t, false, st)) != MSDA_OK) return s;
    ForwardPlan f{};
    if (tc || pieces) {
        f = forward_plan(p, pieces ? 1 : 2);
        a.splits = f.splits, a.tiles_per_split = f.per;
    } else {
        simt_splits(dt, p, &a.splits, &a.tiles_per_split);
    }
    if (a.splits > 1) {
        unsigned char* part = static_cast<unsigned char*>(workspace) + ms.bytes;
        a.part_o = reinterpret_cast<float*>(part);
        a.part_lse = reinterpret_cast<float*>(part + up((size_t)a.splits * p->B * p->M * p->Q * p->D * 4));
    }
    if (pieces) {
        if ((s = msda::error_word(&a.err)) != MSDA_OK) return s;
        unsigned char* ws = static_cast<unsigned char*>(workspace) + ms.bytes + part_bytes(p, a.splits);
        if ((s = make_pieces(a, p, nullptr, ws, st)) != MSDA_OK) return s;
        const PieceSpace w = piece_space(p, false);
        CUtensorMap mq, mk, mv;
        if (!piece_map(p, ws + w.q, f.G, p->Q, p->N, f.qpt, &mq) || !piece_map(p, ws + w.k, 1, p->S, p->N, msda::kTcRows, &mk) ||
            !piece_map(p, ws + w.v, 1, p->S, p->N, msda::kTcRows, &mv))
            return failf(MSDA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
        t.a = a;
        t.G = f.G, t.qpt = f.qpt, t.rows = f.G * f.qpt, t.qblocks = f.qblocks;
        msda::TraceSpan ts(st);
        cudaError_t e = msda::launch_attention_tc_f32(t, mq, mk, mv, st);
        a.tiles_per_split *= 2;  // of 64 keys
        if (e == cudaSuccess) e = msda::launch_attention_simt<float>(a, simt_vec(a), st);
        s = launched(e, "attention kernel launch");
        ts.end(MSDA_KERNEL_ATTENTION, p->B * p->M * p->Q);
    } else if (tc) {
        if ((s = msda::error_word(&a.err)) != MSDA_OK) return s;
        CUtensorMap mq, mk, mv;
        if (!rows_map(dt, query, p->D, f.G, p->Q, p->N, p->B, a.q_sb, a.q_ss, a.q_sh, f.qpt, &mq) ||
            !rows_map(dt, key, p->D, 1, p->S, p->N, p->B, a.k_sb, a.k_ss, a.k_sh, msda::kTcRows, &mk) ||
            !rows_map(dt, value, p->D, 1, p->S, p->N, p->B, a.v_sb, a.v_ss, a.v_sh, msda::kTcRows, &mv))
            return failf(MSDA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
        t.a = a;
        t.G = f.G, t.qpt = f.qpt, t.rows = f.G * f.qpt, t.qblocks = f.qblocks;
        msda::TraceSpan ts(st);
        s = launched(msda::launch_attention_tc_forward(t, dt == MSDA_BF16, f.nq, mq, mk, mv, st), "attention kernel launch");
        ts.end(MSDA_KERNEL_ATTENTION, p->B * p->M * p->Q);
    } else {
        msda::TraceSpan ts(st);
        s = launched(MSDA_BY_DTYPE(dt, launch_attention_simt, a, simt_vec(a), st), "attention kernel launch");
        ts.end(MSDA_KERNEL_ATTENTION, p->B * p->M * p->Q);
    }
    return s == MSDA_OK && a.splits > 1 ? join_parts(dt, a, p, st) : s;
}

msda_status msda_attention_backward(msda_dtype dt, unsigned flags, const msda_attention_problem* p, double scale,
                                    const void* query, const void* key, const void* value, const uint8_t* key_mask,
                                    const uint8_t* mask, const void* out, const float* lse, const void* grad_out,
                                    void* grad_query, void* grad_key, void* grad_value, void* workspace,
                                    size_t workspace_bytes, msda_stream_t stream) {
    msda::clear_error();
    msda_status s = check(dt, flags, p);
    if (s != MSDA_OK) return s;
    if (!(scale > 0.0 && scale < 1e30)) return failf(MSDA_ERR_INVALID_ARG, "scale=%g must be positive", scale);
    const size_t es = dt == MSDA_F32 ? 4 : 2;
    const bool rows = p->B > 0 && p->Q > 0, keys = p->B > 0 && p->S > 0, both = rows && keys;
    if ((s = msda::need_ptr(query, both, es, "query")) || (s = msda::need_ptr(key, both, es, "key")) ||
        (s = msda::need_ptr(value, both, es, "value")) || (s = msda::need_ptr(out, both, es, "out")) ||
        (s = msda::need_ptr(lse, both, 4, "lse")) || (s = msda::need_ptr(grad_out, both, es, "grad_out")) ||
        (s = msda::need_ptr(grad_query, rows, es, "grad_query")) ||
        (s = msda::need_ptr(grad_key, keys, es, "grad_key")) ||
        (s = msda::need_ptr(grad_value, keys, es, "grad_value")) || (s = masks_ok(flags, p, key_mask, mask)))
        return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!both) {  // nothing to attend to: the gradients are zero
        cudaError_t e = cudaSuccess;
        if (rows) e = cudaMemsetAsync(grad_query, 0, (size_t)p->B * p->Q * p->M * p->D * es, st);
        if (keys && e == cudaSuccess) e = cudaMemsetAsync(grad_key, 0, (size_t)p->B * p->S * p->N * p->D * es, st);
        if (keys && e == cudaSuccess) e = cudaMemsetAsync(grad_value, 0, (size_t)p->B * p->S * p->N * p->D * es, st);
        return launched(e, "cudaMemsetAsync");
    }
    const bool tc = tc_type(dt, p) && tma_rows(query, p->query_stride, p->B, p->Q, p->M) &&
                    tma_rows(key, p->key_stride, p->B, p->S, p->N) && tma_rows(value, p->value_stride, p->B, p->S, p->N) &&
                    msda::aligned_to(grad_out, 16) && msda::aligned_to(grad_query, 16) && msda::aligned_to(grad_key, 16) &&
                    msda::aligned_to(grad_value, 16);
    const size_t need = msda_attention_backward_workspace_size(dt, flags, p);
    const bool pieces = tc_pieces(dt, p, true);
    const BackwardLayout w = backward_layout(dt, flags, p, tc || pieces);
    if (!workspace || workspace_bytes < need || !msda::aligned_to(workspace, 256))
        return failf(MSDA_ERR_WORKSPACE, "workspace of %zu bytes, 256-byte aligned, needed (got %zu)", need,
                     workspace_bytes);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    AttentionArgs a = args_of(flags, p, scale, query, key, value, key_mask, mask);
    a.dout = grad_out, a.dq = grad_query, a.dk = grad_key, a.dv = grad_value;
    float* l2 = reinterpret_cast<float*>(ws + w.l2);
    float* dl = l2 + w.rows.rt;
    a.row_l2 = l2, a.row_dl = dl;
    msda::TcArgs t{};
    if ((s = make_mask(a, mask_space(flags, p, tc || pieces), ws + w.mask, t, tc || pieces, st)) != MSDA_OK) return s;
    {
        msda::TraceSpan ts(st);
        const bool half = tc && dt == MSDA_F16;
        float* top = half ? reinterpret_cast<float*>(ws + w.top) : nullptr;
        t.scale_in = top;
        cudaError_t e = half ? cudaMemsetAsync(top, 0, 8, st) : cudaSuccess;
        if (e == cudaSuccess)
            e = MSDA_BY_DTYPE(dt, launch_attention_prepare, a, w.rows, out, lse, half ? msda::kHalfScale : 0.f, l2, top,
                              tc && msda::aligned_to(out, 16), st);
        s = launched(e, "attention statistics kernel launch");
        ts.end(MSDA_KERNEL_ATTENTION_PREPARE, p->B * p->M * p->Q);
        if (s != MSDA_OK) return s;
    }
    if (tc) {
        if ((s = msda::error_word(&a.err)) != MSDA_OK) return s;
        CUtensorMap mq, mk, mv, mg;
        const int64_t row = p->M * p->D;
        if (!rows_map(dt, query, p->D, 1, p->Q, p->M, p->B, a.q_sb, a.q_ss, a.q_sh, msda::kTcRows, &mq) ||
            !rows_map(dt, key, p->D, 1, p->S, p->N, p->B, a.k_sb, a.k_ss, a.k_sh, msda::kTcRows, &mk) ||
            !rows_map(dt, value, p->D, 1, p->S, p->N, p->B, a.v_sb, a.v_ss, a.v_sh, msda::kTcRows, &mv) ||
            !rows_map(dt, grad_out, p->D, 1, p->Q, p->M, p->B, p->Q * row, row, p->D, msda::kTcRows, &mg))
            return failf(MSDA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
        t.a = a;
        t.G = 1, t.qpt = t.rows = msda::kTcRows, t.qblocks = w.rows.tiles;
        t.fix_rows = a.causal && p->Q > p->S;
        t.delta_out = dl;
        {   // the query kernel first: it leaves delta of rows with one tile of keys for the other
            msda::TraceSpan ts(st);
            s = launched(msda::launch_attention_tc_grad_query(t, dt == MSDA_BF16, mq, mk, mv, mg, st),
                         "attention query gradient kernel launch");
            ts.end(MSDA_KERNEL_ATTENTION_GRAD_QUERY, p->B * p->M * p->Q);
            if (s != MSDA_OK) return s;
        }
        msda::TraceSpan ts(st);
        s = launched(msda::launch_attention_tc_grad_key(t, dt == MSDA_BF16, mq, mk, mv, mg, st),
                     "attention key gradient kernel launch");
        ts.end(MSDA_KERNEL_ATTENTION_GRAD_KEY, p->B * p->N * p->S);
        return s;
    }
    if (pieces) {
        if ((s = msda::error_word(&a.err)) != MSDA_OK) return s;
        unsigned char* at = ws + w.pieces;
        if ((s = make_pieces(a, p, lse, at, st)) != MSDA_OK) return s;
        const PieceSpace x = piece_space(p, true);
        CUtensorMap mq, mk, mv, mg;
        if (!piece_map(p, at + x.q, 1, p->Q, p->M, msda::kTcRows, &mq) || !piece_map(p, at + x.k, 1, p->S, p->N, msda::kTcRows, &mk) ||
            !piece_map(p, at + x.v, 1, p->S, p->N, msda::kTcRows, &mv) || !piece_map(p, at + x.g, 1, p->Q, p->M, msda::kTcRows, &mg))
            return failf(MSDA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
        t.a = a;
        t.G = 1, t.qpt = t.rows = msda::kTcRows, t.qblocks = w.rows.tiles;
        {
            msda::TraceSpan ts(st);
            cudaError_t e = msda::launch_attention_tc_f32_grad_key(t, mq, mk, mv, mg, st);
            if (e == cudaSuccess) e = msda::launch_attention_simt_grad_key<float>(a, w.rows, simt_vec(a), st);
            s = launched(e, "attention key gradient kernel launch");
            ts.end(MSDA_KERNEL_ATTENTION_GRAD_KEY, p->B * p->N * p->S);
            if (s != MSDA_OK) return s;
        }
        msda::TraceSpan ts(st);
        cudaError_t e = msda::launch_attention_tc_f32_grad_query(t, mq, mk, mv, mg, st);
        if (e == cudaSuccess) e = msda::launch_attention_simt_grad_query<float>(a, w.rows, simt_vec(a), st);
        ts.end(MSDA_KERNEL_ATTENTION_GRAD_QUERY, p->B * p->M * p->Q);
        return launched(e, "attention query gradient kernel launch");
    }
    {
        msda::TraceSpan ts(st);
        s = launched(MSDA_BY_DTYPE(dt, launch_attention_simt_grad_key, a, w.rows, simt_vec(a), st),
                     "attention key gradient kernel launch");
        ts.end(MSDA_KERNEL_ATTENTION_GRAD_KEY, p->B * p->N * p->S);
        if (s != MSDA_OK) return s;
    }
    msda::TraceSpan ts(st);
    s = launched(MSDA_BY_DTYPE(dt, launch_attention_simt_grad_query, a, w.rows, simt_vec(a), st),
                 "attention query gradient kernel launch");
    ts.end(MSDA_KERNEL_ATTENTION_GRAD_QUERY, p->B * p->M * p->Q);
    return s;
}

}  // extern "C"
