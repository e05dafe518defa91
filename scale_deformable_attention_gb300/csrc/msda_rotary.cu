// msda_rotary.cu -- host side of msda_norm_rotary_forward / _backward:
// checks, choice of the element or vector form, launches.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdio>

#include "msda_host.cuh"
#include "msda_rotary.cuh"

namespace {

using msda::RotaryArgs;

// Blocks of 256 threads, persistent; the partial sums of the weights'
// gradients have one row a block.
constexpr int kRotaryMaxGrid = msda::kPlanSms * 6;
constexpr int kChunkTokens[] = {32, 16, 8, 4};

// Element form, tokens a chunk: as many as leave two chunks an SM, 32 at most
// (the angles of a chunk are worked out before its rows are read, so a small
// call wants many small chunks and a large one few).
int chunk_tokens(int64_t B, int64_t S) {
    for (int t : kChunkTokens)
        if (B * ((S + t - 1) / t) >= 2 * msda::kPlanSms) return t;
    return 4;
}

msda_status check(msda_dtype dt, unsigned flags, const msda_rotary_problem* p) {
    using msda::failf;
    if (dt != MSDA_F32 && dt != MSDA_F16 && dt != MSDA_BF16) return failf(MSDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
    if (flags & ~(MSDA_ROTARY_INTERLEAVED | MSDA_ROTARY_INVERSE)) return failf(MSDA_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    if (!p) return failf(MSDA_ERR_INVALID_ARG, "problem is NULL");
    if (p->B < 0 || p->S < 0 || p->M < 0 || p->N < 0 || p->D < 0 || p->axes < 0)
        return failf(MSDA_ERR_INVALID_ARG, "negative size (B=%lld S=%lld M=%lld N=%lld D=%lld axes=%lld)", (long long)p->B,
                     (long long)p->S, (long long)p->M, (long long)p->N, (long long)p->D, (long long)p->axes);
    if (p->D > msda::kRotaryMaxChannels)
        return failf(MSDA_ERR_UNSUPPORTED, "D=%lld above %d", (long long)p->D, msda::kRotaryMaxChannels);
    if (p->axes < 1 || p->axes > msda::kRotaryMaxAxes)
        return failf(MSDA_ERR_UNSUPPORTED, "axes=%lld outside 1..%d", (long long)p->axes, msda::kRotaryMaxAxes);
    int64_t pairs = 0;
    for (int a = 0; a < p->axes; ++a) {
        if (p->section[a] < 0 || p->section[a] > p->D)
            return failf(MSDA_ERR_INVALID_ARG, "section[%d]=%lld outside 0..D", a, (long long)p->section[a]);
        pairs += p->section[a];
    }
    if (2 * pairs > p->D)
        return failf(MSDA_ERR_INVALID_ARG, "%lld rotated pairs need %lld channels, D=%lld", (long long)pairs,
                     (long long)(2 * pairs), (long long)p->D);
    if (p->position_type < 0 || p->position_type > 2)
        return failf(MSDA_ERR_INVALID_ARG, "unknown position type %lld", (long long)p->position_type);
    if (p->S > INT32_MAX - 64 || p->M > 65536 || p->N > 65536)
        return failf(MSDA_ERR_UNSUPPORTED, "S=%lld, M=%lld or N=%lld too large", (long long)p->S, (long long)p->M,
                     (long long)p->N);
    int64_t t;
    if (!msda::mul_fits(p->B, p->S, &t) || !msda::mul_fits(t, p->M + p->N + 1, &t) ||
        !msda::mul_fits(t, (p->D + p->axes) * 8, &t))
        return failf(MSDA_ERR_INVALID_ARG, "B*S*(M+N)*D overflows 64 bits");
    for (int i = 0; i < 3; ++i)
        if (p->query_stride[i] < 0 || p->key_stride[i] < 0)
            return failf(MSDA_ERR_INVALID_ARG, "negative stride");
    if (p->position_stride < 0) return failf(MSDA_ERR_INVALID_ARG, "negative stride");
    return MSDA_OK;
}

bool vectors_fit(size_t es, const void* x, const int64_t* stride, const void* y, const void* dy, const void* w) {
    for (int i = 0; i < 3; ++i)
        if ((stride[i] * (int64_t)es) % 16) return false;
    return msda::aligned_to(x, 16) && msda::aligned_to(y, 16) && msda::aligned_to(dy, 16) && msda::aligned_to(w, 16);
}

msda_status run(msda_dtype dt, unsigned flags, const msda_rotary_problem* p, double eps, const void* pos,
                const float* freq, const void* q, const void* k, const void* wq, const void* wk, const void* gq,
                const void* gk, void* oq, void* ok, void* dwq, void* dwk, bool norm, bool bwd, void* ws,
                size_t ws_bytes, cudaStream_t st) {
    using msda::failf;
    const size_t es = dt == MSDA_F32 ? 4 : 2;
    int64_t pairs = 0;
    RotaryArgs a{};
    for (int i = 0; i < p->axes; ++i) {
        pairs += p->section[i];
        a.axis_end[i] = (int)pairs;
    }
    const int64_t rows = p->B * p->S;
    const bool any = rows > 0 && p->D > 0 && (p->M > 0 || p->N > 0);
    msda_status s = MSDA_OK;
    const struct { const void* p; bool need; size_t al; const char* name; } ptrs[] = {
        {pos, any && pairs > 0, (size_t)(p->position_type == 2 ? 8 : 4), "positions"},
        {freq, any && pairs > 0, 4, "frequencies"},
        {q, any && p->M > 0, es, "query"},
        {k, any && p->N > 0, es, "key"},
        {oq, any && p->M > 0, es, bwd ? "grad_query" : "query_out"},
        {ok, any && p->N > 0, es, bwd ? "grad_key" : "key_out"},
        {wq, norm && any && p->M > 0, es, "query_weight"},
        {wk, norm && any && p->N > 0, es, "key_weight"},
        {gq, bwd && any && p->M > 0, es, "grad_query_out"},
        {gk, bwd && any && p->N > 0, es, "grad_key_out"},
        {dwq, bwd && p->D > 0 && p->M > 0, es, "grad_query_weight"},
        {dwk, bwd && p->D > 0 && p->N > 0, es, "grad_key_weight"},
    };
    for (const auto& c : ptrs)
        if ((s = msda::need_ptr(c.p, c.need, c.al, c.name)) != MSDA_OK) return s;
    if (!any) {
        if (bwd && p->D > 0) {  // nothing to sum: the weights' gradients are zero
            cudaError_t e = cudaSuccess;
            if (p->M > 0) e = cudaMemsetAsync(dwq, 0, p->D * es, st);
            if (e == cudaSuccess && p->N > 0) e = cudaMemsetAsync(dwk, 0, p->D * es, st);
            if (e != cudaSuccess) return msda::failf(MSDA_ERR_CUDA, "cudaMemsetAsync: %s", cudaGetErrorString(e));
        }
        return MSDA_OK;
    }
    if (bwd) {
        const size_t need = msda_norm_rotary_backward_workspace_size(p);
        if (!ws || ws_bytes < need || !msda::aligned_to(ws, 16))
            return failf(MSDA_ERR_WORKSPACE, "workspace of %zu bytes, 16-byte aligned, needed (got %zu)", need, ws_bytes);
    }
    a.t[0] = {q, gq, oq, norm ? wq : nullptr, p->query_stride[0], p->query_stride[1], p->query_stride[2], (int)p->M};
    a.t[1] = {k, gk, ok, norm ? wk : nullptr, p->key_stride[0], p->key_stride[1], p->key_stride[2], (int)p->N};
    a.pos = pos;
    a.freq = freq;
    a.partial = static_cast<float*>(ws);
    a.pos_sb = p->position_stride;
    a.pos_type = (int)p->position_type;
    a.S = (int)p->S, a.D = (int)p->D, a.P = (int)pairs, a.A = (int)p->axes;
    a.T = chunk_tokens(p->B, p->S);
    a.chunks_per_b = (int)((p->S + a.T - 1) / a.T);
    a.chunks = p->B * a.chunks_per_b;
    a.eps = (float)eps;
    a.inv_d = 1.f / (float)p->D;
    a.sign = (flags & MSDA_ROTARY_INVERSE) ? -1.f : 1.f;
    const bool inter = (flags & MSDA_ROTARY_INTERLEAVED) != 0;
    const int V = (int)(16 / es);
    // 16-byte vectors where every row is made of them (and, in halves, both
    // halves of the pairs) and a row takes no more lanes than a warp has
    const bool fit = p->D % V == 0 && p->D / V <= 32 && (inter || pairs % V == 0) &&
                     (p->M == 0 || vectors_fit(es, q, p->query_stride, oq, gq, wq)) &&
                     (p->N == 0 || vectors_fit(es, k, p->key_stride, ok, gk, wk));
    int mode = msda::ROT_SCALAR, lg = 0;
    size_t smem = (size_t)a.T * a.P * sizeof(float2);
    int64_t blocks = a.chunks;
    if (fit) {
        mode = inter ? msda::ROT_INTERLEAVED : msda::ROT_HALVES;
        while ((1 << lg) < p->D / V) ++lg;
        // a warp takes all heads of its tokens, so that an angle is worked out
        // once, unless that leaves fewer than 16 warps an SM
        a.tokens = rows;
        const int64_t groups = (rows + (32 >> lg) - 1) / (32 >> lg), heads = p->M + p->N;
        int64_t parts = (msda::kPlanSms * 16 + groups - 1) / groups;
        if (parts > heads) parts = heads;
        a.per = (int)((heads + parts - 1) / parts);
        a.parts = (int)((heads + a.per - 1) / a.per);
        smem = 0;
        const int warps = msda::kRotaryThreads / 32;
        blocks = (groups * a.parts + warps - 1) / warps;
    }
    if (bwd && smem < (size_t)(msda::kRotaryThreads / 32) * a.D * 4) smem = (size_t)(msda::kRotaryThreads / 32) * a.D * 4;
    const int64_t most = bwd ? kRotaryMaxGrid : (int64_t)1 << 30;
    const unsigned grid = (unsigned)(blocks < most ? blocks : most);
    cudaError_t e;
    {
        msda::TraceSpan ts(st);
        e = dt == MSDA_F32   ? msda::launch_rotary<float>(a, mode, norm, bwd, lg, inter, grid, smem, st)
            : dt == MSDA_F16 ? msda::launch_rotary<__half>(a, mode, norm, bwd, lg, inter, grid, smem, st)
                             : msda::launch_rotary<__nv_bfloat16>(a, mode, norm, bwd, lg, inter, grid, smem, st);
        ts.end(bwd ? MSDA_KERNEL_ROTARY_BACKWARD : MSDA_KERNEL_ROTARY, rows * (p->M + p->N));
    }
    if (e != cudaSuccess) return failf(MSDA_ERR_CUDA, "rotary kernel launch: %s", cudaGetErrorString(e));
    if (bwd) {
        msda::TraceSpan ts(st);
        void* wk_out = p->N > 0 ? dwk : nullptr;
        void* wq_out = p->M > 0 ? dwq : nullptr;
        e = dt == MSDA_F32   ? msda::launch_rotary_weight<float>(a.partial, (int)grid, a.D, wq_out, wk_out, st)
            : dt == MSDA_F16 ? msda::launch_rotary_weight<__half>(a.partial, (int)grid, a.D, wq_out, wk_out, st)
                             : msda::launch_rotary_weight<__nv_bfloat16>(a.partial, (int)grid, a.D, wq_out, wk_out, st);
        ts.end(MSDA_KERNEL_CONVERT, 2 * p->D);
        if (e != cudaSuccess) return failf(MSDA_ERR_CUDA, "rotary weight kernel launch: %s", cudaGetErrorString(e));
    }
    return MSDA_OK;
}

}  // namespace

extern "C" {

size_t msda_norm_rotary_backward_workspace_size(const msda_rotary_problem* p) {
    if (!p || p->B <= 0 || p->S <= 0 || p->D <= 0 || p->D > msda::kRotaryMaxChannels) return 0;
    return (size_t)kRotaryMaxGrid * 2 * (size_t)p->D * 4;
}

msda_status msda_norm_rotary_forward(msda_dtype dt, unsigned flags, const msda_rotary_problem* problem, double eps,
                                     const void* positions, const float* frequencies, const void* query,
                                     const void* key, const void* query_weight, const void* key_weight,
                                     void* query_out, void* key_out, msda_stream_t stream) {
    msda::clear_error();
    msda_status s = check(dt, flags, problem);
    if (s != MSDA_OK) return s;
    const bool norm = query_weight || key_weight;
    if (norm && !(eps >= 0.0 && eps < 1e30)) return msda::failf(MSDA_ERR_INVALID_ARG, "eps=%g is not a non-negative number", eps);
    return run(dt, flags, problem, eps, positions, frequencies, query, key, query_weight, key_weight, nullptr, nullptr,
               query_out, key_out, nullptr, nullptr, norm, false, nullptr, 0, reinterpret_cast<cudaStream_t>(stream));
}

msda_status msda_norm_rotary_backward(msda_dtype dt, unsigned flags, const msda_rotary_problem* problem, double eps,
                                      const void* positions, const float* frequencies, const void* query,
                                      const void* key, const void* query_weight, const void* key_weight,
                                      const void* grad_query_out, const void* grad_key_out, void* grad_query,
                                      void* grad_key, void* grad_query_weight, void* grad_key_weight, void* workspace,
                                      size_t workspace_bytes, msda_stream_t stream) {
    msda::clear_error();
    msda_status s = check(dt, flags, problem);
    if (s != MSDA_OK) return s;
    if (!(eps >= 0.0 && eps < 1e30)) return msda::failf(MSDA_ERR_INVALID_ARG, "eps=%g is not a non-negative number", eps);
    if (flags & MSDA_ROTARY_INVERSE)
        return msda::failf(MSDA_ERR_INVALID_ARG, "MSDA_ROTARY_INVERSE is for msda_norm_rotary_forward");
    return run(dt, flags, problem, eps, positions, frequencies, query, key, query_weight, key_weight, grad_query_out,
               grad_key_out, grad_query, grad_key, grad_query_weight, grad_key_weight, true, true, workspace,
               workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
