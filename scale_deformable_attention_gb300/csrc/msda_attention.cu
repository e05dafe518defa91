// msda_attention.cu -- host side of msda_attention_forward / _backward:
// checks, workspace layout, choice of kernels, launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "msda_attention.cuh"
#include "msda_attention_simt.cuh"
#include "msda_host.cuh"

namespace msda {

// Keys that some query of the heads sharing them may see, as bytes
// [LB][LN][S] (cleared before): a key outside it may hold anything, NaN too.
// Blocks of 256 keys and 64 queries; every writer writes the same 1.
__global__ void __launch_bounds__(256) msda_attention_live_kernel(const uint8_t* mask, long long mk_sb, long long mk_sh,
                                                                  long long mk_sq, const uint8_t* key_mask,
                                                                  long long km_sb, int Q, int S, int G, int LB, int LN,
                                                                  int heads, uint8_t* live) {
    const int j = blockIdx.x * 256 + threadIdx.x;
    if (j >= S) return;
    for (int z = blockIdx.z; z < LB * LN; z += gridDim.z) {
        const int lb = z / LN, ln = z - lb * LN;
        bool any = false;
        for (int q0 = blockIdx.y * 64; q0 < Q && !any; q0 += gridDim.y * 64) {
            const int q1 = min(Q, q0 + 64);
            for (int h = 0; h < heads && !any; ++h) {
                const uint8_t* p = mask + lb * mk_sb + (long long)(ln * G + h) * mk_sh + q0 * mk_sq + j;
#pragma unroll 8
                for (int q = q0; q < q1; ++q, p += mk_sq) any |= *p != 0;
            }
        }
        if (any && (!key_mask || key_mask[lb * km_sb + j])) live[(long long)z * S + j] = 1;
    }
}

}  // namespace msda

namespace {

using msda::AttentionArgs;
using msda::AttentionRows;
using msda::failf;

constexpr int kSms = 152;  // SMs that a grid is sized for

constexpr unsigned kFlags = MSDA_ATTENTION_CAUSAL | MSDA_ATTENTION_KEY_MASK | MSDA_ATTENTION_MASK;

size_t up(size_t n) { return (n + 255) / 256 * 256; }

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

// Workspace of the liveness of keys under a mask: [LB][LN][S] bytes.
struct Live {
    int LB = 1, LN = 1, heads = 1;
    size_t bytes = 0;
};
Live live_of(unsigned flags, const msda_attention_problem* p) {
    Live l;
    if (!(flags & MSDA_ATTENTION_MASK)) return l;
    l.LB = (flags & MSDA_ATTENTION_KEY_MASK) || (p->B > 1 && p->mask_stride[0] != 0) ? (int)p->B : 1;
    l.LN = p->M > 1 && p->mask_stride[1] != 0 ? (int)p->N : 1;
    l.heads = l.LN > 1 || (p->N == 1 && p->M > 1 && p->mask_stride[1] != 0) ? (int)(p->M / p->N) : 1;
    l.bytes = up((size_t)l.LB * l.LN * (size_t)p->S);
    return l;
}

// Split of the key axis of the FMA-pipe forward: enough blocks for four a SM,
// so that a single query over a long key axis uses the whole GPU.
void simt_splits(const msda_attention_problem* p, int* splits, int* per) {
    const int64_t blocks = p->B * p->M * ((p->Q + 63) / 64), tiles = (p->S + 63) / 64;
    int64_t n = 1;
    if (blocks > 0 && blocks < 2 * kSms && tiles > 1) {
        n = (4 * kSms + blocks - 1) / blocks;
        if (n > tiles) n = tiles;
        if (n > 64) n = 64;
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
    a.c2 = (float)(scale * 1.4426950408889634);
    a.splits = 1;
    a.tiles_per_split = 1 << 30;
    return a;
}

// Replaces key_mask by the keys that some pair of the mask leaves.
msda_status make_live(AttentionArgs& a, const Live& l, void* ws, cudaStream_t st) {
    if (!a.mask || a.S == 0 || a.B == 0) return MSDA_OK;
    uint8_t* live = static_cast<uint8_t*>(ws);
    msda::TraceSpan ts(st);
    cudaError_t e = cudaMemsetAsync(live, 0, (size_t)l.LB * l.LN * a.S, st);
    if (e == cudaSuccess && a.Q > 0) {
        const int64_t z = (int64_t)l.LB * l.LN, y = (a.Q + 63) / 64;
        const dim3 grid((unsigned)((a.S + 255) / 256), (unsigned)(y < 65535 ? y : 65535), (unsigned)(z < 65535 ? z : 65535));
        msda::msda_attention_live_kernel<<<grid, 256, 0, st>>>(a.mask, a.mk_sb, a.mk_sh, a.mk_sq, a.key_mask, a.km_sb, a.Q,
                                                               a.S, a.G, l.LB, l.LN, l.heads, live);
        e = cudaGetLastError();
    }
    ts.end(MSDA_KERNEL_ATTENTION_MASK, (int64_t)a.Q * a.S);
    if (e != cudaSuccess) return failf(MSDA_ERR_CUDA, "mask kernel launch: %s", cudaGetErrorString(e));
    a.key_mask = live;
    a.km_sb = l.LB > 1 ? (long long)l.LN * a.S : 0;
    a.km_sh = l.LN > 1 ? a.S : 0;
    return MSDA_OK;
}

bool simt_vec(const AttentionArgs& a) {  // binary32 rows read as 16-byte vectors
    const long long st[] = {a.q_sb, a.q_ss, a.q_sh, a.k_sb, a.k_ss, a.k_sh, a.v_sb, a.v_ss, a.v_sh, a.D};
    for (long long s : st)
        if (s % 4) return false;
    return msda::aligned_to(a.q, 16) && msda::aligned_to(a.k, 16) && msda::aligned_to(a.v, 16) &&
           msda::aligned_to(a.dout, 16);
}

#define MSDA_BY_DTYPE(dt, f, ...)                       \
    ((dt) == MSDA_F32   ? msda::f<float>(__VA_ARGS__)   \
     : (dt) == MSDA_F16 ? msda::f<__half>(__VA_ARGS__)  \
                        : msda::f<__nv_bfloat16>(__VA_ARGS__))

msda_status launched(cudaError_t e, const char* what) {
    return e == cudaSuccess ? MSDA_OK : failf(MSDA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

// Workspace of the backward: the rows' statistics, then the keys' liveness.
struct BackwardLayout {
    AttentionRows rows;
    size_t l2 = 0, dl = 0, live = 0, bytes = 0;
};
BackwardLayout backward_layout(unsigned flags, const msda_attention_problem* p) {
    BackwardLayout w;
    w.rows = {64, 64, (int)((p->Q + 63) / 64), (int)p->M, 1};
    const size_t n = up((size_t)p->B * w.rows.N * w.rows.tiles * w.rows.rt * 4);
    w.dl = n;
    w.live = 2 * n;
    w.bytes = 2 * n + live_of(flags, p).bytes;
    return w;
}

}  // namespace

extern "C" {

size_t msda_attention_forward_workspace_size(msda_dtype dt, unsigned flags, const msda_attention_problem* p) {
    if (check(dt, flags, p) != MSDA_OK) return 0;
    int splits, per;
    simt_splits(p, &splits, &per);
    return part_bytes(p, splits) + live_of(flags, p).bytes;
}

size_t msda_attention_backward_workspace_size(msda_dtype dt, unsigned flags, const msda_attention_problem* p) {
    if (check(dt, flags, p) != MSDA_OK) return 0;
    return backward_layout(flags, p).bytes;
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
    if ((s = make_live(a, live_of(flags, p), workspace, st)) != MSDA_OK) return s;
    unsigned char* part = static_cast<unsigned char*>(workspace) + live_of(flags, p).bytes;
    simt_splits(p, &a.splits, &a.tiles_per_split);
    if (a.splits > 1) {
        a.part_o = reinterpret_cast<float*>(part);
        a.part_lse = reinterpret_cast<float*>(part + up((size_t)a.splits * p->B * p->M * p->Q * p->D * 4));
    }
    {
        msda::TraceSpan ts(st);
        s = launched(MSDA_BY_DTYPE(dt, launch_attention_simt, a, simt_vec(a), st), "attention kernel launch");
        ts.end(MSDA_KERNEL_ATTENTION, p->B * p->M * p->Q);
    }
    if (s == MSDA_OK && a.splits > 1) {
        msda::TraceSpan ts(st);
        s = launched(MSDA_BY_DTYPE(dt, launch_attention_join, a, st), "attention join kernel launch");
        ts.end(MSDA_KERNEL_ATTENTION_JOIN, p->B * p->M * p->Q);
    }
    return s;
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
    const BackwardLayout w = backward_layout(flags, p);
    if (!workspace || workspace_bytes < w.bytes || !msda::aligned_to(workspace, 256))
        return failf(MSDA_ERR_WORKSPACE, "workspace of %zu bytes, 256-byte aligned, needed (got %zu)", w.bytes,
                     workspace_bytes);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    AttentionArgs a = args_of(flags, p, scale, query, key, value, key_mask, mask);
    a.dout = grad_out, a.dq = grad_query, a.dk = grad_key, a.dv = grad_value;
    float* l2 = reinterpret_cast<float*>(ws + w.l2);
    float* dl = reinterpret_cast<float*>(ws + w.dl);
    a.row_l2 = l2, a.row_dl = dl;
    if ((s = make_live(a, live_of(flags, p), ws + w.live, st)) != MSDA_OK) return s;
    {
        msda::TraceSpan ts(st);
        s = launched(MSDA_BY_DTYPE(dt, launch_attention_prepare, a, w.rows, out, lse, l2, dl, st),
                     "attention statistics kernel launch");
        ts.end(MSDA_KERNEL_ATTENTION_PREPARE, p->B * p->M * p->Q);
        if (s != MSDA_OK) return s;
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
