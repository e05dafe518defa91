// msda_attention_tc_backward.cu -- gradients of softmax attention on the tensor
// cores (tcgen05, sm_103a), fp16 and bf16, D a multiple of 8 up to 128.
//
//   P = 2^(c S - l2),  dS = P (dP - delta),  dP = dO V^T
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K
//
// Two kernels, each recomputing P: one a tile of 128 keys walking the queries
// (S^T, dP^T, dV, dK: four products), one a tile of 128 queries walking the keys
// (S, dP, dQ: three).  One kernel for all would need five products, not seven,
// but its dQ is summed over blocks: 128 x D binary32 values a pair of tiles
// through the L2's reductions, which take 4.2 TB/s here (14.5 bytes a cycle
// and SM: 4500 cycles for 128 channels, against 1536 for the two products saved),
// in an order that changes from run to run.  These two add in a fixed order.
//
// P^T and dS^T (16 bits) are operands in tensor memory, where a product with D
// columns takes D/2 cycles (from shared memory it is bound by reading its
// 128 x 16 operand: 32 + D/4).  Both are written over the scores they come from.
// f16 would lose small values: P is scaled by 2^14 (kHalfScale) and dS by a power of two that the
// largest norms of dO and V rows bound from above; the sums are scaled back.
#include "msda_attention_tc.cuh"
#include "msda_attention_tc_host.cuh"
#include "msda_host.cuh"

namespace msda {

// Warpgroups on the scores, beside one of copies, products and clearing.  Up to
// 64 channels four, 32 columns of a tile each: two left half of the cycles to
// waits.  Beyond, where the products bound the kernel, two of 64 columns: four
// measured the same.
constexpr int bwd_groups(int nc) { return nc == 1 ? 4 : 2; }
constexpr int bwd_threads(int nc) { return bwd_groups(nc) * 128 + 128; }

// Exponents of the scalings: P 2^kp and dS 2^ks.
struct TcScale {
    float ds, inv_p, inv_ds;  // 2^(ks - kp); 2^-kp; 2^-ks (kp is within the rows' l2)
};
template <bool BF16>
__device__ __forceinline__ TcScale tc_scale(const TcArgs& p) {
    TcScale r{1.f, 1.f, 1.f};
    if constexpr (!BF16) {
        // |dS| <= 2 |dO row| |v row|: the power of two that brings this to 2^15 at most (f16 holds 65504)
        const float top = 2.f * sqrtf(p.scale_in[0]) * sqrtf(p.scale_in[1]);
        int ks = 0;
        if (top > 0.f && top < 1e30f) ks = 15 - (int)ceilf(log2f(top));
        ks = ks < -40 ? -40 : ks > 40 ? 40 : ks;
        r.ds = exp2f(ks - kHalfScale);
        r.inv_p = exp2f(-kHalfScale);
        r.inv_ds = exp2f((float)-ks);
    }
    return r;
}

struct TcBackwardSync {
    uint64_t own, full[8], empty[8], ready[8];
    uint64_t s_full[2], dp_full, dp_free, p_ready[2], ds_ready[2], ds_done[2], cleared, acc, delta;
    uint32_t tmem, abort;
    uint32_t words[8][4];
};

// ---- gradients of keys and values ----

template <int NC>
struct TcKeyCfg {
    static constexpr int kStages = NC == 1 ? 4 : 2;  // Q, dO and the rows' statistics
    static constexpr uint32_t kTileBytes = NC * kTcTile;
    static constexpr uint32_t kStatBytes = 1024;
    static constexpr size_t kSmem = 2 * kTileBytes + kStages * (2 * kTileBytes + kStatBytes) + 1024;
    // Tensor memory.  Up to 64 channels there is room for S twice: dS then lies beside P over
    // its S, so dP's columns are free once read, S is made two tiles ahead and dP one, and the
    // products go to two warps (scores; gradients).  One warp had five waits, four commits and
    // 24 products a tile to issue, 2380 cycles one behind the other, while nothing else was
    // busy for half of them.  Beyond, P lies over S, dS over dP, and one warp issues all: its
    // order then stands for barriers.
    static constexpr bool kAhead = NC == 1;
    static constexpr uint32_t kDP = kAhead ? 256 : 128, kDV = kAhead ? 384 : 256, kDK = kAhead ? 448 : 384;
};

template <bool BF16, int NC>
__global__ void __launch_bounds__(bwd_threads(NC), 1)
    msda_attention_tc_grad_key_kernel(const TcArgs p, const __grid_constant__ CUtensorMap map_q,
                                      const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                                      const __grid_constant__ CUtensorMap map_do) {
    using Cfg = TcKeyCfg<NC>;
    constexpr int ST = Cfg::kStages;
    constexpr uint32_t kStage = 2 * Cfg::kTileBytes;
    const AttentionArgs& a = p.a;
    extern __shared__ unsigned char tc_smem_raw[];
    unsigned char* smem = tc_smem_raw + ((1024u - (tc_smem(tc_smem_raw) & 1023u)) & 1023u);  // stays a shared-memory address to the compiler
    unsigned char* k_tile = smem;
    unsigned char* v_tile = smem + Cfg::kTileBytes;
    unsigned char* ring = smem + 2 * Cfg::kTileBytes;                      // Q, dO a stage
    float* stats = reinterpret_cast<float*>(ring + ST * kStage);  // l2[128], delta[128] a stage (signs turned: ready to add)
    __shared__ TcBackwardSync sy;
    constexpr int NG = bwd_groups(NC), CH = 4 / NG;  // warpgroups, parts of 32 columns each
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int ktiles = (a.S + kTcRows - 1) / kTcRows;
    long long id = blockIdx.x;
    const int kt = (int)(id % ktiles);  // causal: the keys that most queries see come first
    id /= ktiles;
    const int n = (int)(id % a.N), b = (int)(id / a.N);
    const int j0 = kt * kTcRows;
    const uint8_t* km = a.key_mask ? a.key_mask + b * a.km_sb + n * a.km_sh : nullptr;
    // row tiles that see a key of the tile: causal rows below j0 - (S - Q) see none
    long long first_q = a.causal ? (long long)j0 - (a.S - a.Q) : 0;
    int r0 = first_q <= 0 ? 0 : (int)(first_q < a.Q ? first_q / kTcRows : p.qblocks), r1 = p.qblocks;
    tc_narrow(p, p.ext_k, ktiles, b, n * a.G, a.G, kt, kt, &r0, &r1);
    int nt = a.G * max(0, r1 - r0);
    if (km) {  // a tile of keys that take no part has no gradients
        const bool any = tid < min(kTcRows, a.S - j0) && km[j0 + tid] != 0;
        if (!__syncthreads_or(any)) nt = 0;
    }

    if (warp == NG * 4) {
        if (lane == 0) {
            for (int i = 0; i < ST; ++i) {
                tc_bar_init(tc_smem(&sy.full[i]), 1);
                tc_bar_init(tc_smem(&sy.empty[i]), 1);
                tc_bar_init(tc_smem(&sy.ready[i]), 1);
            }
            tc_bar_init(tc_smem(&sy.own), 1);
            tc_bar_init(tc_smem(&sy.dp_full), 1);
            tc_bar_init(tc_smem(&sy.dp_free), NG * 4);
            for (int i = 0; i < 2; ++i) {
                tc_bar_init(tc_smem(&sy.s_full[i]), 1);
                tc_bar_init(tc_smem(&sy.p_ready[i]), NG * 4);
                tc_bar_init(tc_smem(&sy.ds_ready[i]), NG * 4);
            }
            tc_bar_init(tc_smem(&sy.acc), 1);
            tc_bar_init(tc_smem(&sy.cleared), 1);
            sy.abort = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    } else if (warp == NG * 4 + 1) {
        tmem_alloc(tc_smem(&sy.tmem), 512);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sy.tmem;
    volatile uint32_t* abort = &sy.abort;
    const bool fix = km || p.fix_rows;  // operands that a warp clears before the products read them
    bool ok = true;

    if (warp < NG * 4) {
        // ---- probabilities and their gradients: thread = key row, CH parts of 32 of a tile's 128 queries ----
        const int w = warp >> 2, wl = warp & 3, row = wl * 32 + lane, j = j0 + row;
        const uint32_t first = lane == 0;
        const uint32_t lanes = (uint32_t)wl << 21;
        const uint32_t dp_at = tmem + Cfg::kDP + w * CH * 32 + lanes;
        const uint64_t c2 = tc_two(a.c2, a.c2);
        const float dscale = tc_scale<BF16>(p).ds;
        const bool has_bits = p.bits_t != nullptr;
        const int shift = a.S - a.Q;
        int g = 0, rt = r0;  // head of the group and row tile of step i
#pragma unroll 1
        for (int i = 0; i < nt; ++i, rt + 1 < r1 ? ++rt : (++g, rt = r0)) {
            const int st = i % ST, q0 = rt * kTcRows + w * CH * 32;
            const int buf = Cfg::kAhead ? i & 1 : 0, phase = (Cfg::kAhead ? i >> 1 : i) & 1;
            const uint32_t s_at = tmem + buf * 128 + w * CH * 32 + lanes;
            uint32_t bw[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                bw[c] = ~0u;
                if (has_bits && j < a.S)
                    bw[c] = p.bits_t[b * p.bits_t_sb + (n * a.G + g) * p.bits_t_sh + (long long)j * p.Wq + rt * 4 + w * CH + c];
            }
            const float* l2 = stats + st * 256 + w * CH * 32;
            const float* dl = l2 + 128;
            ok = tc_bar_wait(tc_smem(&sy.full[st]), (i / ST) & 1, abort, a.err) &&
                 tc_bar_wait(tc_smem(&sy.s_full[buf]), phase, abort, a.err);
            if (!ok) break;
            tc_fence_after();
            uint32_t s[CH][32];
#pragma unroll
            for (int c = 0; c < CH; ++c) tmem_ld32(s[c], s_at + c * 32);
            tmem_wait_ld();
            // P^T over the thread's own columns of S^T
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                // causal: query q sees key j if q >= j - shift
                if (a.causal) bw[c] &= ~tc_low_bits(j - shift - q0 - c * 32);
                if (__builtin_expect(__any_sync(0xffffffffu, bw[c] != 0xffffffffu), 0)) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (!((bw[c] >> k) & 1u)) s[c][k] = 0xff800000u;
                }
                uint32_t pk[16];
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const float4 l = *reinterpret_cast<const float4*>(l2 + c * 32 + k);
                    float x0, x1, x2, x3;
                    tc_split(tc_fma2(tc_two(__uint_as_float(s[c][k]), __uint_as_float(s[c][k + 1])), c2, tc_two(l.x, l.y)), x0, x1);
                    tc_split(tc_fma2(tc_two(__uint_as_float(s[c][k + 2]), __uint_as_float(s[c][k + 3])), c2, tc_two(l.z, l.w)), x2, x3);
                    const float e0 = tc_ex2(x0), e1 = tc_ex2(x1), e2 = tc_ex2(x2), e3 = tc_ex2(x3);
                    s[c][k] = __float_as_uint(e0), s[c][k + 1] = __float_as_uint(e1);
                    s[c][k + 2] = __float_as_uint(e2), s[c][k + 3] = __float_as_uint(e3);
                    pk[k / 2] = tc_pack<BF16>(e0, e1);
                    pk[k / 2 + 1] = tc_pack<BF16>(e2, e3);
                }
                tmem_st16(s_at + c * 32, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            tc_bar_arrive_if(first, tc_smem(&sy.p_ready[buf]));
            ok = tc_bar_wait(tc_smem(&sy.dp_full), i & 1, abort, a.err);
            if (!ok) break;
            tc_fence_after();
            // dS^T beside P^T, or over dP^T
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                uint32_t d[32], pk[16];
                tmem_ld32(d, dp_at + c * 32);
                tmem_wait_ld();
                if (Cfg::kAhead && c == CH - 1) {
                    tc_fence_before();
                    tc_bar_arrive_if(first, tc_smem(&sy.dp_free));
                }
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const float4 l = *reinterpret_cast<const float4*>(dl + c * 32 + k);
                    float x0, x1, x2, x3;
                    uint64_t y0 = tc_add2(tc_two(__uint_as_float(d[k]), __uint_as_float(d[k + 1])), tc_two(l.x, l.y));
                    uint64_t y1 = tc_add2(tc_two(__uint_as_float(d[k + 2]), __uint_as_float(d[k + 3])), tc_two(l.z, l.w));
                    y0 = tc_mul2(y0, tc_two(__uint_as_float(s[c][k]), __uint_as_float(s[c][k + 1])));
                    y1 = tc_mul2(y1, tc_two(__uint_as_float(s[c][k + 2]), __uint_as_float(s[c][k + 3])));
                    if constexpr (!BF16) y0 = tc_mul2(y0, tc_two(dscale, dscale)), y1 = tc_mul2(y1, tc_two(dscale, dscale));
                    tc_split(y0, x0, x1);
                    tc_split(y1, x2, x3);
                    pk[k / 2] = tc_pack<BF16>(x0, x1);
                    pk[k / 2 + 1] = tc_pack<BF16>(x2, x3);
                }
                tmem_st16(Cfg::kAhead ? s_at + c * 32 + 16 : dp_at + c * 32, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            // (two tiles ahead: a barrier a buffer, as a warp may be a tile ahead of another)
            tc_bar_arrive_if(first, tc_smem(&sy.ds_ready[buf]));
        }
        // ---- dV (the first half of the warpgroups) and dK, in chunks of 16 channels ----
        if (nt > 0 && ok) {
            ok = tc_bar_wait(tc_smem(&sy.acc), 0, abort, a.err);
            tc_fence_after();
        }
        if (ok) {
            const bool live = nt > 0 && j < a.S && (!km || km[j]);
            const TcScale sc = tc_scale<BF16>(p);
            const bool is_v = w < NG / 2;
            const float f = is_v ? sc.inv_p : sc.inv_ds * a.scale;
            const uint32_t at = tmem + (is_v ? Cfg::kDV : Cfg::kDK) + lanes;
            unsigned char* out = static_cast<unsigned char*>(is_v ? a.dv : a.dk) + (((long long)b * a.S + j) * a.N + n) * a.D * 2;
            for (int c = w % (NG / 2); c < (a.D + 15) / 16; c += NG / 2) {
                uint32_t o[16];
                if (nt > 0) {
                    tmem_ld16(o, at + c * 16);
                    tmem_wait_ld();
                }
                if (j >= a.S) continue;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = live ? tc_pack<BF16>(__uint_as_float(o[8 * k + 2 * e]) * f, __uint_as_float(o[8 * k + 2 * e + 1]) * f) : 0u;
                    if (c * 16 + 8 * k < a.D) reinterpret_cast<uint4*>(out + c * 32)[k] = make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
        }
    } else {
        const int role = warp - NG * 4;
        uint64_t* full = fix ? sy.ready : sy.full;
        if (role == 0 && nt > 0) {
            // ---- copies ----
            const uint32_t on = tc_elect(), own = tc_smem(&sy.own);
            tc_bar_expect_if(on, own, 2 * Cfg::kTileBytes);
            for (int c = 0; c < NC; ++c) {
                tc_tma_5d_if(on, tc_smem(k_tile) + c * kTcTile, &map_k, own, c * 64, j0, n, b);
                tc_tma_5d_if(on, tc_smem(v_tile) + c * kTcTile, &map_v, own, c * 64, j0, n, b);
            }
            int g = 0, rt = r0;
            const float* stat = a.row_l2 + ((long long)b * a.M + n * a.G) * p.qblocks * 256;
            for (int i = 0; i < nt; ++i, rt + 1 < r1 ? ++rt : (++g, rt = r0)) {
                const int st = i % ST, h = n * a.G + g;
                if (i >= ST) ok = tc_bar_wait(tc_smem(&sy.empty[st]), (i / ST - 1) & 1, abort, a.err);
                if (!ok) break;
                const uint32_t bar = tc_smem(&sy.full[st]), at = tc_smem(ring) + st * kStage;
                tc_bar_expect_if(on, bar, kStage + Cfg::kStatBytes);
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    tc_tma_5d_if(on, at + c * kTcTile, &map_q, bar, c * 64, rt * kTcRows, h, b);
                    tc_tma_5d_if(on, at + Cfg::kTileBytes + c * kTcTile, &map_do, bar, c * 64, rt * kTcRows, h, b);
                }
                tc_bulk_if(on, tc_smem(stats) + st * 1024, stat + ((long long)g * p.qblocks + rt) * 256, 1024, bar);
            }
        } else if ((role == 1 || (Cfg::kAhead && role == 3)) && nt > 0) {
            // ---- products ----
            const uint32_t on = tc_elect();
            const int steps = (a.D + 15) / 16;
            const uint32_t id_s = tc_idesc(BF16, false, false, 128, 128), id_g = tc_idesc(BF16, false, true, 128, steps * 16);
            const uint64_t k_desc = tc_desc(tc_smem(k_tile), 16, 1024), v_desc = tc_desc(tc_smem(v_tile), 16, 1024);
            const uint32_t base = tc_smem(ring);
            // stage of step i: Q, and dO a tile further
            const uint64_t row_desc = tc_desc(base, 16, 1024), col_desc = tc_desc(base, kTcTile, 1024);
            auto off = [&](int i) { return (uint64_t)((i % ST) * (kStage >> 4)); };
            constexpr uint64_t kToDo = Cfg::kTileBytes >> 4;
            auto filled = [&](int i) { return tc_bar_wait(tc_smem(&full[i % ST]), (i / ST) & 1, abort, a.err); };
            // 128 keys x 128 queries: into d, with y the tile of queries (or of their gradients)
            auto scores = [&](uint32_t d, uint64_t x_desc, uint64_t y_desc, uint32_t bar) {
#pragma unroll
                for (int k = 0; k < NC * 4; ++k) {
                    const uint64_t o = ((k >> 2) * kTcTile + (k & 3) * 32) >> 4;
                    if (k < steps) tc_mma_ss(on, d, x_desc + o, y_desc + o, id_s, k > 0);
                }
                tc_commit(on, bar);
            };
            // sums over the tile's queries
            auto gradient = [&](uint32_t d, uint32_t x, uint64_t y_desc, bool acc) {
#pragma unroll
                for (int k = 0; k < 8; ++k)  // 16 queries; the warpgroups' parts of 32 lie 32 columns apart
                    tc_mma_ts(on, d, x + (k >> 1) * 32 + (k & 1) * 8, y_desc + ((k * 2048) >> 4), id_g, acc || k > 0);
            };
            const uint32_t dp = tmem + Cfg::kDP, dv_at = tmem + Cfg::kDV, dk_at = tmem + Cfg::kDK;
            if (role == 1) {
                ok = tc_bar_wait(tc_smem(&sy.own), 0, abort, a.err);
                if (ok && fix) ok = tc_bar_wait(tc_smem(&sy.cleared), 0, abort, a.err);
                ok = ok && filled(0);
                if (ok) {
                    tc_fence_after();
                    scores(tmem, k_desc, row_desc + off(0), tc_smem(&sy.s_full[0]));
                    scores(dp, v_desc, row_desc + off(0) + kToDo, tc_smem(&sy.dp_full));
                }
            }
            if constexpr (Cfg::kAhead) {
                if (role == 1) {
                    if (ok && nt > 1) {
                        ok = filled(1);
                        tc_fence_after();
                        if (ok) scores(tmem + 128, k_desc, row_desc + off(1), tc_smem(&sy.s_full[1]));
                    }
                    for (int i = 0; i + 1 < nt && ok; ++i) {
                        ok = tc_bar_wait(tc_smem(&sy.dp_free), i & 1, abort, a.err);
                        if (!ok) break;
                        tc_fence_after();
                        scores(dp, v_desc, row_desc + off(i + 1) + kToDo, tc_smem(&sy.dp_full));
                        if (i + 2 < nt) {  // over S(i), when P(i) and dS(i) are used up
                            ok = filled(i + 2) && tc_bar_wait(tc_smem(&sy.empty[i % ST]), (i / ST) & 1, abort, a.err);
                            if (!ok) break;
                            tc_fence_after();
                            scores(tmem + (i & 1) * 128, k_desc, row_desc + off(i + 2), tc_smem(&sy.s_full[i & 1]));
                        }
                    }
                } else {
                    for (int i = 0; i < nt; ++i) {
                        const int buf = i & 1, phase = (i >> 1) & 1;
                        ok = tc_bar_wait(tc_smem(&sy.p_ready[buf]), phase, abort, a.err);
                        if (!ok) break;
                        tc_fence_after();
                        gradient(dv_at, tmem + buf * 128, col_desc + off(i) + kToDo, i > 0);
                        ok = tc_bar_wait(tc_smem(&sy.ds_ready[buf]), phase, abort, a.err);
                        if (!ok) break;
                        tc_fence_after();
                        gradient(dk_at, tmem + buf * 128 + 16, col_desc + off(i), i > 0);
                        tc_commit(on, tc_smem(&sy.empty[i % ST]));
                    }
                    if (ok) tc_commit(on, tc_smem(&sy.acc));
                }
            } else {
                for (int i = 0; i < nt && ok; ++i) {
                    ok = tc_bar_wait(tc_smem(&sy.p_ready[0]), i & 1, abort, a.err);
                    if (!ok) break;
                    tc_fence_after();
                    gradient(dv_at, tmem, col_desc + off(i) + kToDo, i > 0);
                    if (i + 1 < nt) {
                        ok = filled(i + 1);
                        if (!ok) break;
                        tc_fence_after();
                        scores(tmem, k_desc, row_desc + off(i + 1), tc_smem(&sy.s_full[0]));
                    }
                    ok = tc_bar_wait(tc_smem(&sy.ds_ready[0]), i & 1, abort, a.err);
                    if (!ok) break;
                    tc_fence_after();
                    gradient(dk_at, dp, col_desc + off(i), i > 0);
                    tc_commit(on, tc_smem(&sy.empty[i % ST]));
                    if (i + 1 < nt) scores(dp, v_desc, row_desc + off(i + 1) + kToDo, tc_smem(&sy.dp_full));
                }
                if (ok) tc_commit(on, tc_smem(&sy.acc));
            }
        } else if (role == 2 && fix && nt > 0) {
            // ---- keys, and rows without keys, that take no part ----
            ok = tc_bar_wait(tc_smem(&sy.own), 0, abort, a.err);
            if (ok) {
                if (km) {
                    uint32_t w[4];
                    tc_key_words(km + j0, a.S - j0, lane, w);
                    tc_clear_rows<NC>(k_tile, w, lane);
                    tc_clear_rows<NC>(v_tile, w, lane);
                    tc_fence_async();
                }
                __syncwarp();
                if (lane == 0) tc_bar_arrive(tc_smem(&sy.cleared));
            }
            for (int i = 0; i < nt && ok; ++i) {
                const int st = i % ST;
                ok = tc_bar_wait(tc_smem(&sy.full[st]), (i / ST) & 1, abort, a.err);
                if (!ok) break;
                uint32_t w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    w[c] = __ballot_sync(0xffffffffu, stats[st * 256 + c * 32 + lane] != -attn_inf());
                if ((w[0] & w[1] & w[2] & w[3]) != 0xffffffffu) {
                    tc_clear_rows<NC>(ring + st * kStage, w, lane);
                    tc_clear_rows<NC>(ring + st * kStage + Cfg::kTileBytes, w, lane);
                    tc_fence_async();
                }
                __syncwarp();
                if (lane == 0) tc_bar_arrive(tc_smem(&sy.ready[st]));
            }
        }
        __syncwarp();
    }
    if (!ok) tc_drain();
    tc_fence_before();
    __syncthreads();
    if (warp == NG * 4 + 1) tmem_dealloc(tmem, 512);
}

// ---- gradient of queries ----

template <int NC>
struct TcQueryCfg {
    // Up to 64 channels: stages of K and V, S two tiles ahead, dP one, dS over its S, the
    // products on two warps (as in the key kernel).  Beyond: a ring of tiles
    // V(0), K(0), V(1), ...; V is let go behind its scores, K behind dQ.
    // (Pairs of K and V in two stages left the products waiting 1600 of 3200
    // cycles a tile for them at 128 channels.)
    static constexpr bool kAhead = NC == 1;
    static constexpr int kRing = NC == 1 ? 8 : 5;  // tiles
    static constexpr uint32_t kTileBytes = NC * kTcTile;
    static constexpr size_t kSmem = (2 + kRing) * kTileBytes + 1024;
    // tensor memory, kAhead: S twice (dS over it), dP, dQ; else S, dP, dS twice (dQ of a tile runs beside the next tile's dS), dQ
    static constexpr uint32_t kDP = kAhead ? 256 : 128, kDS = 256, kDQ = 384;
};

template <bool BF16, int NC>
__global__ void __launch_bounds__(bwd_threads(NC), 1)
    msda_attention_tc_grad_query_kernel(const TcArgs p, const __grid_constant__ CUtensorMap map_q,
                                        const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                                        const __grid_constant__ CUtensorMap map_do) {
    using Cfg = TcQueryCfg<NC>;
    constexpr int R = Cfg::kRing;
    const AttentionArgs& a = p.a;
    extern __shared__ unsigned char tc_smem_raw[];
    unsigned char* smem = tc_smem_raw + ((1024u - (tc_smem(tc_smem_raw) & 1023u)) & 1023u);  // stays a shared-memory address to the compiler
    unsigned char* q_tile = smem;
    unsigned char* do_tile = smem + Cfg::kTileBytes;
    unsigned char* ring = smem + 2 * Cfg::kTileBytes;
    __shared__ TcBackwardSync sy;
    constexpr int NG = bwd_groups(NC), CH = 4 / NG;  // warpgroups, parts of 32 columns each
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    long long id = blockIdx.x;
    int rt = (int)(id % p.qblocks);
    id /= p.qblocks;
    const int h = (int)(id % a.M), b = (int)(id / a.M), n = h / a.G;
    if (a.causal) rt = p.qblocks - 1 - rt;
    const int q0 = rt * kTcRows;
    const uint8_t* km = a.key_mask ? a.key_mask + b * a.km_sb + n * a.km_sh : nullptr;
    int t0 = 0, t1 = (tc_seen(a, min(q0 + kTcRows, a.Q) - 1) + kTcRows - 1) / kTcRows;
    tc_narrow(p, p.ext_q, p.qblocks, b, h, 1, rt, rt, &t0, &t1);
    if (km) tc_trim(km, a.S, &t0, &t1);
    const int nt = max(0, t1 - t0);

    if (warp == NG * 4) {
        if (lane == 0) {
            for (int i = 0; i < R; ++i) {
                tc_bar_init(tc_smem(&sy.full[i]), 1);
                tc_bar_init(tc_smem(&sy.empty[i]), 1);
                tc_bar_init(tc_smem(&sy.ready[i]), 1);
            }
            tc_bar_init(tc_smem(&sy.own), 1);
            tc_bar_init(tc_smem(&sy.acc), 1);
            tc_bar_init(tc_smem(&sy.delta), NG * 4);
            tc_bar_init(tc_smem(&sy.dp_full), 1);
            tc_bar_init(tc_smem(&sy.dp_free), NG * 4);
            for (int i = 0; i < 2; ++i) {
                tc_bar_init(tc_smem(&sy.s_full[i]), 1);
                tc_bar_init(tc_smem(&sy.ds_ready[i]), NG * 4);
                tc_bar_init(tc_smem(&sy.ds_done[i]), 1);
            }
            sy.abort = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    } else if (warp == NG * 4 + 1) {
        tmem_alloc(tc_smem(&sy.tmem), 512);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sy.tmem;
    volatile uint32_t* abort = &sy.abort;
    bool ok = true;

    if (warp < NG * 4) {
        // thread = query row, CH parts of 32 of a tile's 128 keys
        const int w = warp >> 2, wl = warp & 3, row = wl * 32 + lane, q = q0 + row;
        const uint32_t first = lane == 0;
        const uint32_t lanes = (uint32_t)wl << 21;
        const uint32_t dp_at = tmem + Cfg::kDP + w * CH * 32 + lanes;
        const TcScale sc = tc_scale<BF16>(p);
        const long long r = (((long long)b * a.M + h) * p.qblocks + rt) * 256 + row;
        const float l2 = a.row_l2[r], dl = a.row_dl[r];
        const bool live = l2 != -attn_inf();  // q < Q and some key seen
        const int seen = live ? tc_seen(a, q) : 0;
        const int seen_least = __reduce_min_sync(0xffffffffu, live ? seen : a.S);
        const uint32_t* bits = a.bits && q < a.Q ? a.bits + b * a.bits_sb + h * a.bits_sh + (long long)q * a.W : nullptr;
        const uint64_t c2 = tc_two(a.c2, a.c2), nl = tc_two(l2, l2), ds2 = tc_two(sc.ds, sc.ds);
        uint64_t nd = tc_two(dl * sc.ds, dl * sc.ds);
#pragma unroll 1
        for (int i = 0; i < nt; ++i) {
            const int j0 = (t0 + i) * kTcRows + w * CH * 32;
            uint32_t bw[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) bw[c] = bits ? bits[(t0 + i) * 4 + w * CH + c] : ~0u;
            const int buf = i & 1;
            const uint32_t s_at = tmem + (Cfg::kAhead ? buf * 128 : 0) + w * CH * 32 + lanes;
            ok = tc_bar_wait(tc_smem(&sy.s_full[Cfg::kAhead ? buf : 0]), (Cfg::kAhead ? i >> 1 : i) & 1, abort, a.err);
            if (!ok) break;
            tc_fence_after();
            uint32_t s[CH][32], d[CH][32];
#pragma unroll
            for (int c = 0; c < CH; ++c) tmem_ld32(s[c], s_at + c * 32);
            if constexpr (!Cfg::kAhead) {
#pragma unroll
                for (int c = 0; c < CH; ++c) tmem_ld32(d[c], dp_at + c * 32);
            }
            tmem_wait_ld();
            if constexpr (!Cfg::kAhead) {  // both are read: the next may be made
                tc_fence_before();
                tc_bar_arrive_if(first, tc_smem(&sy.dp_free));
            }
            if (__builtin_expect(km || a.bits || seen_least - j0 < CH * 32, 0)) {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    bw[c] &= tc_low_bits(seen - j0 - c * 32);
                    if (km) bw[c] &= sy.words[i & 7][w * CH + c];
                    if (__any_sync(0xffffffffu, bw[c] != 0xffffffffu)) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!((bw[c] >> k) & 1u)) s[c][k] = 0xff800000u;
                    }
                }
            }
            auto probability = [&](int c, int k) {
                float x0, x1;
                tc_split(tc_fma2(tc_two(__uint_as_float(s[c][k]), __uint_as_float(s[c][k + 1])), c2, nl), x0, x1);
                return tc_two(tc_ex2(x0), tc_ex2(x1));
            };
            if constexpr (Cfg::kAhead) {  // while dP is on its way
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        float e0, e1;
                        tc_split(probability(c, k), e0, e1);
                        s[c][k] = __float_as_uint(e0), s[c][k + 1] = __float_as_uint(e1);
                    }
                ok = tc_bar_wait(tc_smem(&sy.dp_full), i & 1, abort, a.err);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < CH; ++c) tmem_ld32(d[c], dp_at + c * 32);
                tmem_wait_ld();
                tc_fence_before();
                tc_bar_arrive_if(first, tc_smem(&sy.dp_free));
            } else if (i > 1) {  // dS(i-2) is used up
                ok = tc_bar_wait(tc_smem(&sy.ds_done[buf]), (i / 2 - 1) & 1, abort, a.err);
                if (!ok) break;
                tc_fence_after();
            }
            if (nt == 1) {
                // All keys that the tile's rows see are in this one: delta = sum_j p dP from the values at hand, not <dout, out>.
                // With few keys out is as large as a value and its rounding to 16 bits, carried into dP - delta, was the
                // largest error (twice the others together for two keys).
                float2* part_sum = reinterpret_cast<float2*>(ring + 2 * Cfg::kTileBytes);  // one tile: the ring's third is free
                float sum = 0.f, ps = 0.f;
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int k = 0; k < 32; ++k) {  // a pair that takes no part adds nothing, whatever its dP
                        float e = __uint_as_float(s[c][k]);
                        if (!Cfg::kAhead) e = tc_ex2(fmaf(e, a.c2, l2));
                        if (e != 0.f) sum = fmaf(e, __uint_as_float(d[c][k]), sum), ps += e;
                    }
                part_sum[w * 128 + row] = make_float2(sum, ps);
                __syncwarp();
                if (lane == 0) tc_bar_arrive(tc_smem(&sy.delta));
                ok = tc_bar_wait(tc_smem(&sy.delta), 0, abort, a.err);
                if (!ok) break;
                sum = ps = 0.f;
#pragma unroll
                for (int g = 0; g < NG; ++g) sum += part_sum[g * 128 + row].x, ps += part_sum[g * 128 + row].y;
                // over the probabilities' own sum, which their rounding keeps off 1: the row's dS then add up to 0
                const float delta = live && ps > 0.f ? -sum / ps : 0.f;
                nd = tc_two(delta * sc.ds, delta * sc.ds);
                if (w == 0) p.delta_out[r] = delta;
            }
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    float x0, x1;
                    const uint64_t e = Cfg::kAhead ? tc_two(__uint_as_float(s[c][k]), __uint_as_float(s[c][k + 1])) : probability(c, k);
                    const uint64_t dp = tc_two(__uint_as_float(d[c][k]), __uint_as_float(d[c][k + 1]));
                    tc_split(tc_mul2(BF16 ? tc_add2(dp, nd) : tc_fma2(dp, ds2, nd), e), x0, x1);
                    pk[k / 2] = tc_pack<BF16>(x0, x1);
                }
                tmem_st16(Cfg::kAhead ? s_at + c * 32 : tmem + Cfg::kDS + buf * 64 + (w * CH + c) * 16 + lanes, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            // one barrier a buffer: a warp may be a tile ahead of another, and its arrival must not count for that other's
            tc_bar_arrive_if(first, tc_smem(&sy.ds_ready[buf]));
        }
        if (nt > 0 && ok) {
            ok = tc_bar_wait(tc_smem(&sy.acc), 0, abort, a.err);
            tc_fence_after();
        }
        if (ok) {  // the warpgroups take chunks of 16 channels in turn
            const float f = sc.inv_ds * a.scale;
            unsigned char* out = static_cast<unsigned char*>(a.dq) + (((long long)b * a.Q + q) * a.M + h) * a.D * 2;
            for (int c = w; c < (a.D + 15) / 16; c += NG) {
                uint32_t o[16];
                if (nt > 0) {
                    tmem_ld16(o, tmem + Cfg::kDQ + lanes + c * 16);
                    tmem_wait_ld();
                }
                if (q >= a.Q) continue;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = live && nt > 0 ? tc_pack<BF16>(__uint_as_float(o[8 * k + 2 * e]) * f, __uint_as_float(o[8 * k + 2 * e + 1]) * f) : 0u;
                    if (c * 16 + 8 * k < a.D) reinterpret_cast<uint4*>(out + c * 32)[k] = make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
        }
    } else {
        const int role = warp - NG * 4;
        uint64_t* full = km ? sy.ready : sy.full;
        // kAhead: stage i holds K and V in tiles 2i and 2i + 1 of the ring, under one barrier (that of the even tile);
        // else V(i) is tile 2i, K(i) tile 2i + 1, each with its own
        constexpr int ST = R / 2;
        if (role == 0 && nt > 0) {
            // ---- copies ----
            const uint32_t on = tc_elect(), own = tc_smem(&sy.own);
            tc_bar_expect_if(on, own, 2 * Cfg::kTileBytes);
            for (int c = 0; c < NC; ++c) {
                tc_tma_5d_if(on, tc_smem(q_tile) + c * kTcTile, &map_q, own, c * 64, q0, h, b);
                tc_tma_5d_if(on, tc_smem(do_tile) + c * kTcTile, &map_do, own, c * 64, q0, h, b);
            }
            if constexpr (Cfg::kAhead) {
                for (int i = 0; i < nt; ++i) {
                    const int st = 2 * (i % ST);
                    if (i >= ST) ok = tc_bar_wait(tc_smem(&sy.empty[st]), (i / ST - 1) & 1, abort, a.err);
                    if (!ok) break;
                    const uint32_t bar = tc_smem(&sy.full[st]), at = tc_smem(ring) + st * Cfg::kTileBytes;
                    tc_bar_expect_if(on, bar, 2 * Cfg::kTileBytes);
                    tc_tma_5d_if(on, at, &map_k, bar, 0, (t0 + i) * kTcRows, n, b);
                    tc_tma_5d_if(on, at + Cfg::kTileBytes, &map_v, bar, 0, (t0 + i) * kTcRows, n, b);
                }
            } else {
                for (int x = 0, st = 0, wrap = 0; x < 2 * nt; ++x) {
                    if (x >= R) ok = tc_bar_wait(tc_smem(&sy.empty[st]), (wrap - 1) & 1, abort, a.err);
                    if (!ok) break;
                    const uint32_t bar = tc_smem(&sy.full[st]), at = tc_smem(ring) + st * Cfg::kTileBytes;
                    tc_bar_expect_if(on, bar, Cfg::kTileBytes);
#pragma unroll
                    for (int c = 0; c < NC; ++c)
                        tc_tma_5d_if(on, at + c * kTcTile, (x & 1) ? &map_k : &map_v, bar, c * 64, (t0 + (x >> 1)) * kTcRows, n, b);
                    if (++st == R) st = 0, ++wrap;
                }
            }
        } else if ((role == 1 || role == 3) && nt > 0) {
            // ---- products: scores, and dQ ----
            const uint32_t on = tc_elect();
            const int steps = (a.D + 15) / 16;
            const uint32_t id_s = tc_idesc(BF16, false, false, 128, 128), id_g = tc_idesc(BF16, false, true, 128, steps * 16);
            const uint64_t q_desc = tc_desc(tc_smem(q_tile), 16, 1024), do_desc = tc_desc(tc_smem(do_tile), 16, 1024);
            const uint32_t base = tc_smem(ring), dp = tmem + Cfg::kDP;
            const uint64_t row_desc = tc_desc(base, 16, 1024), col_desc = tc_desc(base, kTcTile, 1024);
            constexpr uint64_t kTile = Cfg::kTileBytes >> 4;
            auto scores = [&](uint32_t d, uint64_t x_desc, uint64_t y_desc) {  // 128 queries x 128 keys
#pragma unroll
                for (int k = 0; k < NC * 4; ++k) {
                    const uint64_t o = ((k >> 2) * kTcTile + (k & 3) * 32) >> 4;
                    if (k < steps) tc_mma_ss(on, d, x_desc + o, y_desc + o, id_s, k > 0);
                }
            };
            // dQ += dS K over the tile's keys: 16 a step, a warpgroup's part of 32 `part` columns behind the one before
            auto gradient = [&](uint32_t x, uint32_t part, uint64_t y_desc, bool acc) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    tc_mma_ts(on, tmem + Cfg::kDQ, x + (k >> 1) * part + (k & 1) * 8, y_desc + ((k * 2048) >> 4), id_g, acc || k > 0);
            };
            if constexpr (Cfg::kAhead) {
                auto off = [&](int i) { return 2 * (i % ST) * kTile; };
                auto filled = [&](int i) { return tc_bar_wait(tc_smem(&full[2 * (i % ST)]), (i / ST) & 1, abort, a.err); };
                if (role == 1) {
                    ok = tc_bar_wait(tc_smem(&sy.own), 0, abort, a.err) && filled(0);
                    if (ok) {
                        tc_fence_after();
                        scores(tmem, q_desc, row_desc);
                        tc_commit(on, tc_smem(&sy.s_full[0]));
                        scores(dp, do_desc, row_desc + kTile);
                        tc_commit(on, tc_smem(&sy.dp_full));
                    }
                    if (ok && nt > 1) {
                        ok = filled(1);
                        tc_fence_after();
                        if (ok) {
                            scores(tmem + 128, q_desc, row_desc + off(1));
                            tc_commit(on, tc_smem(&sy.s_full[1]));
                        }
                    }
                    for (int i = 0; i + 1 < nt && ok; ++i) {
                        ok = tc_bar_wait(tc_smem(&sy.dp_free), i & 1, abort, a.err);
                        if (!ok) break;
                        tc_fence_after();
                        scores(dp, do_desc, row_desc + off(i + 1) + kTile);
                        tc_commit(on, tc_smem(&sy.dp_full));
                        if (i + 2 < nt) {  // over S(i), when dS(i) is used up
                            ok = filled(i + 2) && tc_bar_wait(tc_smem(&sy.empty[2 * (i % ST)]), (i / ST) & 1, abort, a.err);
                            if (!ok) break;
                            tc_fence_after();
                            scores(tmem + (i & 1) * 128, q_desc, row_desc + off(i + 2));
                            tc_commit(on, tc_smem(&sy.s_full[i & 1]));
                        }
                    }
                } else {
                    for (int i = 0; i < nt; ++i) {
                        ok = tc_bar_wait(tc_smem(&sy.ds_ready[i & 1]), (i >> 1) & 1, abort, a.err);
                        if (!ok) break;
                        tc_fence_after();
                        gradient(tmem + (i & 1) * 128, 32, col_desc + off(i), i > 0);
                        tc_commit(on, tc_smem(&sy.empty[2 * (i % ST)]));
                    }
                    if (ok) tc_commit(on, tc_smem(&sy.acc));
                }
            } else {
                if (role == 1) {
                    ok = tc_bar_wait(tc_smem(&sy.own), 0, abort, a.err);
                    for (int i = 0, sv = 0, pv = 0; i < nt && ok; ++i) {  // slot and phase of V(i), then of K(i)
                        const int sk = sv + 1 == R ? 0 : sv + 1, pk = sk == 0 ? pv ^ 1 : pv;
                        ok = tc_bar_wait(tc_smem(&full[sv]), pv, abort, a.err) && tc_bar_wait(tc_smem(&full[sk]), pk, abort, a.err) &&
                             (i == 0 || tc_bar_wait(tc_smem(&sy.dp_free), (i - 1) & 1, abort, a.err));
                        if (!ok) break;
                        tc_fence_after();
                        scores(dp, do_desc, row_desc + sv * kTile);
                        tc_commit(on, tc_smem(&sy.empty[sv]));
                        scores(tmem, q_desc, row_desc + sk * kTile);
                        tc_commit(on, tc_smem(&sy.s_full[0]));
                        sv = sk + 1 == R ? 0 : sk + 1;
                        pv = sv == 0 ? pk ^ 1 : pk;
                    }
                } else {
                    for (int i = 0, sk = 1; i < nt; ++i) {  // slot of K(i)
                        ok = tc_bar_wait(tc_smem(&sy.ds_ready[i & 1]), (i >> 1) & 1, abort, a.err);
                        if (!ok) break;
                        tc_fence_after();
                        gradient(tmem + Cfg::kDS + (i & 1) * 64, 16, col_desc + sk * kTile, i > 0);
                        tc_commit(on, tc_smem(&sy.ds_done[i & 1]));
                        tc_commit(on, tc_smem(&sy.empty[sk]));
                        sk = sk + 2 >= R ? sk + 2 - R : sk + 2;
                    }
                    if (ok) tc_commit(on, tc_smem(&sy.acc));
                }
            }
        } else if (role == 2 && km && nt > 0) {
            // ---- keys that take no part ----
            uint32_t w[4];
            for (int x = 0, st = 0, wrap = 0; x < 2 * nt && ok; ++x) {
                const int i = x >> 1;
                if (!(x & 1)) {
                    tc_key_words(km + (t0 + i) * kTcRows, a.S - (t0 + i) * kTcRows, lane, w);
                    if (lane < 4) sy.words[i & 7][lane] = lane == 0 ? w[0] : lane == 1 ? w[1] : lane == 2 ? w[2] : w[3];
                }
                if (!Cfg::kAhead || !(x & 1)) ok = tc_bar_wait(tc_smem(&sy.full[st]), wrap & 1, abort, a.err);
                if (!ok) break;
                if ((w[0] & w[1] & w[2] & w[3]) != 0xffffffffu) {
                    tc_clear_rows<NC>(ring + st * Cfg::kTileBytes, w, lane);
                    tc_fence_async();
                }
                __syncwarp();
                if (lane == 0 && (!Cfg::kAhead || (x & 1))) tc_bar_arrive(tc_smem(&sy.ready[Cfg::kAhead ? st - 1 : st]));
                if (++st == R) st = 0, ++wrap;
            }
        }
        __syncwarp();
    }
    if (!ok) tc_drain();
    tc_fence_before();
    __syncthreads();
    if (warp == NG * 4 + 1) tmem_dealloc(tmem, 512);
}

// ---- host ----

template <bool BF16, int NC>
static cudaError_t grad_key_go(const TcArgs& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                               const CUtensorMap& g, cudaStream_t st) {
    constexpr size_t smem = TcKeyCfg<NC>::kSmem;
    static SmemSeen seen;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(&msda_attention_tc_grad_key_kernel<BF16, NC>), smem, seen);
    if (e != cudaSuccess) return e;
    const long long grid = (long long)p.a.B * p.a.N * ((p.a.S + kTcRows - 1) / kTcRows);
    msda_attention_tc_grad_key_kernel<BF16, NC><<<(unsigned)grid, bwd_threads(NC), smem, st>>>(p, q, k, v, g);
    return cudaGetLastError();
}
template <bool BF16, int NC>
static cudaError_t grad_query_go(const TcArgs& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                 const CUtensorMap& g, cudaStream_t st) {
    constexpr size_t smem = TcQueryCfg<NC>::kSmem;
    static SmemSeen seen;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(&msda_attention_tc_grad_query_kernel<BF16, NC>), smem, seen);
    if (e != cudaSuccess) return e;
    const long long grid = (long long)p.a.B * p.a.M * p.qblocks;
    msda_attention_tc_grad_query_kernel<BF16, NC><<<(unsigned)grid, bwd_threads(NC), smem, st>>>(p, q, k, v, g);
    return cudaGetLastError();
}

cudaError_t launch_attention_tc_grad_key(const TcArgs& p, bool bf16, const CUtensorMap& q, const CUtensorMap& k,
                                         const CUtensorMap& v, const CUtensorMap& g, cudaStream_t st) {
    if (p.a.D > 64) return bf16 ? grad_key_go<true, 2>(p, q, k, v, g, st) : grad_key_go<false, 2>(p, q, k, v, g, st);
    return bf16 ? grad_key_go<true, 1>(p, q, k, v, g, st) : grad_key_go<false, 1>(p, q, k, v, g, st);
}
cudaError_t launch_attention_tc_grad_query(const TcArgs& p, bool bf16, const CUtensorMap& q, const CUtensorMap& k,
                                           const CUtensorMap& v, const CUtensorMap& g, cudaStream_t st) {
    if (p.a.D > 64) return bf16 ? grad_query_go<true, 2>(p, q, k, v, g, st) : grad_query_go<false, 2>(p, q, k, v, g, st);
    return bf16 ? grad_query_go<true, 1>(p, q, k, v, g, st) : grad_query_go<false, 1>(p, q, k, v, g, st);
}

}  // namespace msda
