// msda_attention_tc_f32.cu -- softmax attention and its gradients for binary32
// tensors of up to 64 channels on the tensor cores (tcgen05, sm_103a).
//
// A binary32 value is the sum of three bf16 values, x = x0 + x1 + x2: x0 its
// upper 16 bits, x1 and x2 what is left, rounded twice (24 bits and more).  A
// product is taken as x1 y1 + x0 y2 + x2 y0 + x0 y1 + x1 y0 + x0 y0; the three
// pieces left out are below 2^-22 |x y|, 2^-24 on average.  The tensor cores cut
// a sum off where it is added to the accumulator (64 times 0.97 of a unit in the
// last place added to 1 leaves 1), so the small products go first: at the size
// of the result only x0 y0 is cut, one step per 16 values contracted.  For the
// same reason no sum over tiles stays in tensor memory: each tile's products
// start anew, and the threads add them up in registers, rounded.
//
// Six bf16 products of 128 x 128 x 16 take 384 cycles, on the FMA pipe that
// step takes 2048.  64 heads of 48, 900 queries and keys, a mask of pairs:
// forward 350 us on the FMA pipe, 129 here and 16 to cut the tensors; key
// gradient 585 and 160, query gradient 485 and 140 (and 21 to cut).  4096 x 4096
// of 8 heads of 64: 239, 338 and 282 us.  What bounds them: exponentials and
// cutting (11 operations a pair of values) in turn with the products of one tile, as
// 48 KB a tile of an operand leave room for one block and three to four tiles an
// SM, and copies of 96 KB a step.  Pieces let go one by one, and two warpgroups
// on alternate key tiles in the forward, measured the same or worse: a wait and
// a commit more per piece, and 2600 cycles of 3000 for a tile's products then
// stood behind the threads that share their issue slots.
//
// A first kernel cuts the tensors into pieces [3][B, rows, heads, Dp] in the
// workspace, whatever their strides and D, with rows that take no part as
// zeros.  A value beyond 2^60 (an infinity and NaN too) cannot be cut so that
// its products come out as they should (inf * 0): it sets a flag by which these
// kernels return and those of the FMA pipe, launched behind them, run; without
// it those return.
#include "msda_attention_tc.cuh"
#include "msda_attention_tc_host.cuh"
#include "msda_host.cuh"

namespace msda {

namespace {

constexpr uint32_t kPieces = 3 * kTcTile;  // bytes of 128 rows of up to 64 channels in three pieces
// products of pieces, smallest first
constexpr int kPairs = 6;
__device__ constexpr int kPairA[kPairs] = {1, 0, 2, 0, 1, 0}, kPairB[kPairs] = {1, 2, 0, 1, 0, 0};

// The pieces of two finite values, side by side.
__device__ __forceinline__ void pieces(float x, float y, uint32_t& p0, uint32_t& p1, uint32_t& p2) {
    const uint64_t minus = tc_two(-1.f, -1.f);
    p0 = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
    const uint64_t r = tc_fma2(tc_two(__uint_as_float(p0 << 16), __uint_as_float(p0 & 0xffff0000u)), minus, tc_two(x, y));
    tc_split(r, x, y);
    p1 = tc_pack<true>(x, y);
    tc_split(tc_fma2(tc_two(__uint_as_float(p1 << 16), __uint_as_float(p1 & 0xffff0000u)), minus, r), x, y);
    p2 = tc_pack<true>(x, y);
}
// 16 values' pieces into tensor memory, 8 columns each at a, b and c
__device__ __forceinline__ void store_pieces(const float* v, uint32_t a, uint32_t b, uint32_t c) {
    uint32_t p[3][8];
#pragma unroll
    for (int k = 0; k < 8; ++k) pieces(v[2 * k], v[2 * k + 1], p[0][k], p[1][k], p[2][k]);
    tmem_st8(a, p[0]);
    tmem_st8(b, p[1]);
    tmem_st8(c, p[2]);
}

}  // namespace

// Cuts eight channels a thread.  blockIdx.y: the tensor.  Reads a tensor once and writes
// 1.5 times its bytes.
__global__ void __launch_bounds__(256) msda_attention_split_kernel(const SplitArgs a) {
    const SplitTensor t = a.t[blockIdx.y];
    const int vecs = a.Dp / 8;
    const long long rows = (long long)a.B * t.rows * t.heads, total = rows * vecs;
    bool odd = false;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
        const long long row = i / vecs;
        const int c = (int)(i - row * vecs) * 8;
        const long long bs = row / t.heads, b = bs / t.rows;
        const int h = (int)(row - bs * t.heads);
        const long long s = bs - b * t.rows;
        bool on = true;
        if (t.alive) on = t.alive[b * t.alive_sb + h * t.alive_sh + s] != 0;
        if (t.lse) on = t.lse[(b * t.heads + h) * t.rows + s] != -attn_inf();
        float v[8];
        const float* src = t.src + b * t.sb + s * t.ss + h * t.sh + c;
        if (on && t.vec && c + 8 <= a.D) {
            const float4 x = reinterpret_cast<const float4*>(src)[0], y = reinterpret_cast<const float4*>(src)[1];
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = on && c + k < a.D ? src[k] : 0.f;
        }
        uint32_t p[3][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            odd |= !(fabsf(v[2 * k]) <= 0x1p60f) || !(fabsf(v[2 * k + 1]) <= 0x1p60f);
            pieces(v[2 * k], v[2 * k + 1], p[0][k], p[1][k], p[2][k]);
        }
        uint4* dst = reinterpret_cast<uint4*>(t.dst) + i;
#pragma unroll
        for (int k = 0; k < 3; ++k) dst[k * total] = make_uint4(p[k][0], p[k][1], p[k][2], p[k][3]);
    }
    if (odd) *a.odd = 1;
}

namespace {

// The three pieces of a tile of 128 rows; piece k of batch item b is item k * B + b of the map.
__device__ __forceinline__ void load_pieces(uint32_t on, uint32_t to, const CUtensorMap* map, uint32_t bar, int row, int head,
                                            int b, int B) {
    for (int k = 0; k < 3; ++k) tc_tma_5d_if(on, to + k * kTcTile, map, bar, 0, row, head, k * B + b);
}

// d (128 x 128) = X Y^T over up to 64 channels; x, y: descriptors of the first pieces
__device__ __forceinline__ void products_nt(const uint32_t (&step_on)[4], uint32_t d, uint64_t x, uint64_t y, uint32_t idesc) {
#pragma unroll
    for (int e = 0; e < kPairs; ++e)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            tc_mma_ss(step_on[k], d, x + ((kPairA[e] * kTcTile + k * 32) >> 4), y + ((kPairB[e] * kTcTile + k * 32) >> 4), idesc,
                      e > 0 || k > 0);
}

// Adds NC chunks of 16 columns to a thread's sums; chunks from `steps` on hold nothing.
template <int NC>
__device__ __forceinline__ void add_columns(float (&sum)[NC * 16], uint32_t at, int steps) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (c >= steps) break;
        uint32_t x[16];
        tmem_ld16(x, at + c * 16);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) sum[c * 16 + k] += __uint_as_float(x[k]);
    }
}
// N values of a row from channel c0 on, times f
template <int N>
__device__ __forceinline__ void store_columns(float* row, const float (&v)[N], int c0, int D, float f, bool zero) {
    const bool vec = D % 4 == 0 && (reinterpret_cast<uintptr_t>(row) & 15) == 0;
#pragma unroll
    for (int k = 0; k < N; k += 4) {
        const float x[4] = {zero ? 0.f : v[k] * f, zero ? 0.f : v[k + 1] * f, zero ? 0.f : v[k + 2] * f, zero ? 0.f : v[k + 3] * f};
        const int c = c0 + k;
        if (vec) {
            if (c < D) *reinterpret_cast<float4*>(row + c) = make_float4(x[0], x[1], x[2], x[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < D) row[c + e] = x[e];
        }
    }
}

}  // namespace

// ---- forward: a tile of 128 rows of a key head a block (heads that share it side by side) ----

struct TcF32Forward {
    static constexpr int kRing = 3;  // tiles K(0), V(0), K(1), ...
    static constexpr size_t kSmem = (1 + kRing) * kPieces + 1024;
    static constexpr uint32_t kP = 256, kO = 448;  // tensor memory: S twice, P in three pieces of 64, O
};
struct TcF32ForwardSync {
    uint64_t q_full, full[3], empty[3], s_full[2], s_free[2], p_full, pv_done;
    uint32_t tmem, abort;
};

__global__ void __launch_bounds__(256, 1)
    msda_attention_tc_f32_kernel(const TcArgs p, const __grid_constant__ CUtensorMap map_q,
                                 const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
    using Cfg = TcF32Forward;
    constexpr int R = Cfg::kRing;
    const AttentionArgs& a = p.a;
    extern __shared__ unsigned char tc_smem_raw[];
    unsigned char* smem = tc_smem_raw + ((1024u - (tc_smem(tc_smem_raw) & 1023u)) & 1023u);
    unsigned char* q_tile = smem;
    unsigned char* ring = smem + kPieces;
    __shared__ TcF32ForwardSync sy;
    if (*a.odd) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    long long id = blockIdx.x;
    const int split = (int)(id % a.splits);
    id /= a.splits;
    int qb = (int)(id % p.qblocks);
    id /= p.qblocks;
    const int n = (int)(id % a.N), b = (int)(id / a.N);
    if (a.causal) qb = p.qblocks - 1 - qb;
    const int q0 = qb * p.qpt;
    const uint8_t* km = a.key_mask ? a.key_mask + b * a.km_sb + n * a.km_sh : nullptr;
    int t0 = split * a.tiles_per_split;
    int t1 = min(t0 + a.tiles_per_split, (tc_seen(a, min(q0 + p.qpt, a.Q) - 1) + kTcRows - 1) / kTcRows);
    tc_narrow(p, p.ext_q, (a.Q + kTcRows - 1) / kTcRows, b, n * p.G, p.G, q0 / kTcRows, (min(q0 + p.qpt, a.Q) - 1) / kTcRows, &t0, &t1);
    if (km) tc_trim(km, a.S, &t0, &t1);
    const int nt = max(0, t1 - t0);
    if (warp == 4) {
        if (lane == 0) {
            for (int i = 0; i < R; ++i) {
                tc_bar_init(tc_smem(&sy.full[i]), 1);
                tc_bar_init(tc_smem(&sy.empty[i]), 1);
            }
            tc_bar_init(tc_smem(&sy.q_full), 1);
            for (int i = 0; i < 2; ++i) {
                tc_bar_init(tc_smem(&sy.s_full[i]), 1);
                tc_bar_init(tc_smem(&sy.s_free[i]), 4);
            }
            tc_bar_init(tc_smem(&sy.p_full), 4);
            tc_bar_init(tc_smem(&sy.pv_done), 1);
            sy.abort = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    } else if (warp == 5) {
        tmem_alloc(tc_smem(&sy.tmem), 512);
    }
    if (p.rows < kTcRows) {  // rows that no query fills hold zeros
        const uint32_t words = (kTcRows - p.rows) * 8;
        for (uint32_t i = tid; i < 3 * words; i += 256) {
            const uint32_t c = i / words, w = i - c * words;
            *reinterpret_cast<uint4*>(q_tile + c * kTcTile + p.rows * 128 + w * 16) = make_uint4(0, 0, 0, 0);
        }
        tc_fence_async();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sy.tmem;
    volatile uint32_t* abort = &sy.abort;
    bool ok = true;
    if (warp < 4) {
        // ---- softmax: a thread a row, exponentials against the reference at hand (as for 16 bits) ----
        const int row = tid, q = q0 + row / p.G, h = n * p.G + row % p.G;
        const bool valid = row < p.rows && q < a.Q;
        const int seen = valid ? tc_seen(a, q) : 0;
        const int seen_least = __reduce_min_sync(0xffffffffu, valid ? seen : a.S);
        const uint32_t first = lane == 0, lanes = (uint32_t)warp << 21;
        const uint32_t* bits = a.bits && valid ? a.bits + b * a.bits_sb + h * a.bits_sh + (long long)q * a.W : nullptr;
        const uint32_t o_at = tmem + Cfg::kO + lanes, p_at = tmem + Cfg::kP + lanes;
        const int steps = (a.D + 15) / 16;
        float m = -attn_inf(), l = 0.f, o[64];
#pragma unroll
        for (int k = 0; k < 64; ++k) o[k] = 0.f;
#pragma unroll 1
        for (int i = 0; i < nt; ++i) {
            const int j0 = (t0 + i) * kTcRows;
            uint32_t w[4] = {~0u, ~0u, ~0u, ~0u};
            if (km) tc_key_words(km + j0, a.S - j0, lane, w);
            if (bits) {
                const uint4 x = *reinterpret_cast<const uint4*>(bits + (t0 + i) * 4);
                w[0] &= x.x, w[1] &= x.y, w[2] &= x.z, w[3] &= x.w;
            }
            const bool masked = km || a.bits || seen_least - j0 < kTcRows;
            if (masked) {
#pragma unroll
                for (int c = 0; c < 4; ++c) w[c] &= tc_low_bits(seen - j0 - 32 * c);
            }
            ok = tc_bar_wait(tc_smem(&sy.s_full[i & 1]), (i >> 1) & 1, abort, a.err);
            if (!ok) break;
            tc_fence_after();
            const uint32_t s_at = tmem + (i & 1) * 128 + lanes;
            float e[4][32];
            auto scores = [&](int c) {
                tmem_ld32(reinterpret_cast<uint32_t(&)[32]>(e[c]), s_at + c * 32);
                tmem_wait_ld();
                if (masked) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (!((w[c] >> k) & 1u)) e[c][k] = -attn_inf();
                }
            };
            auto probabilities = [&]() {  // 2^(c S - m), and the row's sum of them
                const float ref = m == -attn_inf() ? 0.f : m;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    scores(c);
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        e[c][k] = tc_ex2(fmaf(e[c][k], a.c2, -ref));
                        sum[k & 3] += e[c][k];
                    }
                }
                return (sum[0] + sum[1]) + (sum[2] + sum[3]);
            };
            bool renew = __any_sync(0xffffffffu, valid && m == -attn_inf());
            float sum = 0.f, f = 1.f;
            if (!renew) {
                sum = probabilities();
                renew = __any_sync(0xffffffffu, valid && !(sum <= 16384.f));
            }
            if (renew) {
                float top = -attn_inf();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    scores(c);
#pragma unroll
                    for (int k = 0; k < 32; ++k) top = fmaxf(top, e[c][k]);
                }
                const float next = fmaxf(m, top * a.c2);
                f = next == m ? 1.f : exp2f(m - next);
                m = next;
                l *= f;
                sum = probabilities();
            }
            l += sum;
            tc_fence_before();
            tc_bar_arrive_if(first, tc_smem(&sy.s_free[i & 1]));
            if (i > 0) {  // P(i-1) is used up, and O holds its product
                ok = tc_bar_wait(tc_smem(&sy.pv_done), (i - 1) & 1, abort, a.err);
                if (!ok) break;
                tc_fence_after();
                add_columns<4>(o, o_at, steps);
            }
            if (renew) {
#pragma unroll
                for (int k = 0; k < 64; ++k) o[k] *= f;
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) store_pieces(&e[c >> 1][(c & 1) * 16], p_at + c * 8, p_at + 64 + c * 8, p_at + 128 + c * 8);
            tmem_wait_st();
            tc_fence_before();
            tc_bar_arrive_if(first, tc_smem(&sy.p_full));
        }
        if (nt > 0 && ok) {
            ok = tc_bar_wait(tc_smem(&sy.pv_done), (nt - 1) & 1, abort, a.err);
            tc_fence_after();
            if (ok) add_columns<4>(o, o_at, steps);
        }
        if (ok && valid) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const float l2 = l == 0.f ? -attn_inf() : m + log2f(l);
            const long long r = ((long long)b * a.M + h) * a.Q + q;
            const long long part = (long long)split * a.B * a.M * a.Q + r;
            float* out = a.splits > 1 ? a.part_o + part * a.D : static_cast<float*>(a.out) + (((long long)b * a.Q + q) * a.M + h) * a.D;
            store_columns<64>(out, o, 0, a.D, inv, l == 0.f);
            if (a.splits > 1) a.part_lse[part] = l2;
            else a.lse[r] = l2 * kLn2;
        }
    } else {
        const int role = warp - 4;
        if (role == 0 && nt > 0) {
            const uint32_t on = tc_elect(), qbar = tc_smem(&sy.q_full);
            tc_bar_expect_if(on, qbar, 3 * p.rows * 128);
            load_pieces(on, tc_smem(q_tile), &map_q, qbar, q0, n, b, a.B);
            for (int x = 0; x < 2 * nt; ++x) {
                const int st = x % R;
                if (x >= R) ok = tc_bar_wait(tc_smem(&sy.empty[st]), (x / R - 1) & 1, abort, a.err);
                if (!ok) break;
                const uint32_t bar = tc_smem(&sy.full[st]);
                tc_bar_expect_if(on, bar, kPieces);
                load_pieces(on, tc_smem(ring) + st * kPieces, (x & 1) ? &map_v : &map_k, bar, (t0 + (x >> 1)) * kTcRows, n, b, a.B);
            }
        } else if ((role == 1 || role == 2) && nt > 0) {  // scores; outputs
            const uint32_t on = tc_elect();
            const int steps = (a.D + 15) / 16;
            const uint32_t id_s = tc_idesc(true, false, false, 128, 128), id_o = tc_idesc(true, false, true, 128, steps * 16);
            uint32_t step_on[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) step_on[k] = k < steps ? on : 0u;
            const uint64_t q_desc = tc_desc(tc_smem(q_tile), 16, 1024);
            auto filled = [&](int x) { return tc_bar_wait(tc_smem(&sy.full[x % R]), (x / R) & 1, abort, a.err); };
            if (role == 1) {
                ok = tc_bar_wait(tc_smem(&sy.q_full), 0, abort, a.err);
                for (int i = 0; i < nt && ok; ++i) {
                    ok = filled(2 * i) && (i < 2 || tc_bar_wait(tc_smem(&sy.s_free[i & 1]), ((i >> 1) - 1) & 1, abort, a.err));
                    if (!ok) break;
                    tc_fence_after();
                    products_nt(step_on, tmem + (i & 1) * 128, q_desc, tc_desc(tc_smem(ring) + (2 * i % R) * kPieces, 16, 1024), id_s);
                    tc_commit(on, tc_smem(&sy.s_full[i & 1]));
                    tc_commit(on, tc_smem(&sy.empty[2 * i % R]));
                }
            } else {
                for (int i = 0; i < nt; ++i) {
                    const int x = 2 * i + 1;
                    ok = filled(x) && tc_bar_wait(tc_smem(&sy.p_full), i & 1, abort, a.err);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t v_desc = tc_desc(tc_smem(ring) + (x % R) * kPieces, kTcTile, 1024);
#pragma unroll
                    for (int e = 0; e < kPairs; ++e)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            tc_mma_ts(on, tmem + Cfg::kO, tmem + Cfg::kP + kPairA[e] * 64 + k * 8,
                                      v_desc + ((kPairB[e] * kTcTile + k * 2048) >> 4), id_o, e > 0 || k > 0);
                    tc_commit(on, tc_smem(&sy.pv_done));
                    tc_commit(on, tc_smem(&sy.empty[x % R]));
                }
            }
        }
        __syncwarp();
    }
    if (!ok) tc_drain();
    tc_fence_before();
    __syncthreads();
    if (warp == 5) tmem_dealloc(tmem, 512);
}

// ---- gradients ----

constexpr int kF32Threads = 576;  // four warpgroups on the scores, 32 columns of a tile each; a warp of copies, one of products
struct TcF32BackwardSync {
    uint64_t own, full[2], empty[2], s_full, dp_full, s_free, p_ready, ds_ready;
    uint32_t tmem, abort;
};

namespace {

// Where a warpgroup's three pieces of its 32 columns lie: two over its own columns of `region`, the third 128 columns
// behind, so that none lands on columns that another has still to read.
__device__ __forceinline__ uint32_t piece_column(uint32_t region, int t, int w) {
    return t < 2 ? region + w * 32 + t * 16 : region + 128 + w * 16;
}
// the same for a step of 16 contracted columns (k = 0..7) as an operand
__device__ __forceinline__ uint32_t piece_step(uint32_t region, int t, int k) {
    return t < 2 ? region + (k >> 1) * 32 + t * 16 + (k & 1) * 8 : region + 128 + k * 8;
}
__device__ __forceinline__ void store_pieces_over(uint32_t region, uint32_t lanes, int w, const float (&v)[32]) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
        store_pieces(v + k * 16, piece_column(region, 0, w) + k * 8 + lanes, piece_column(region, 1, w) + k * 8 + lanes,
                     piece_column(region, 2, w) + k * 8 + lanes);
}
// d = (pieces in `region`)(y), y: descriptor of the first piece, rows contracted
__device__ __forceinline__ void products_tn(uint32_t on, uint32_t d, uint32_t region, uint64_t y, uint32_t idesc) {
#pragma unroll
    for (int e = 0; e < kPairs; ++e)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            tc_mma_ts(on, d, piece_step(region, kPairA[e], k), y + ((kPairB[e] * kTcTile + k * 2048) >> 4), idesc, e > 0 || k > 0);
}

}  // namespace

struct TcF32Key {
    static constexpr size_t kSmem = 4 * kPieces + 1024 + 1024;  // K, V, Q, dO; statistics
    static constexpr uint32_t kDP = 192, kDV = 384, kDK = 448;  // tensor memory: S (P over it) 0, dP (dS over it)
};

__global__ void __launch_bounds__(kF32Threads, 1)
    msda_attention_tc_f32_grad_key_kernel(const TcArgs p, const __grid_constant__ CUtensorMap map_q,
                                          const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                                          const __grid_constant__ CUtensorMap map_do) {
    using Cfg = TcF32Key;
    const AttentionArgs& a = p.a;
    extern __shared__ unsigned char tc_smem_raw[];
    unsigned char* smem = tc_smem_raw + ((1024u - (tc_smem(tc_smem_raw) & 1023u)) & 1023u);
    const uint32_t k_tile = tc_smem(smem), v_tile = k_tile + kPieces, q_tile = k_tile + 2 * kPieces, do_tile = k_tile + 3 * kPieces;
    const float* stats = reinterpret_cast<const float*>(smem + 4 * kPieces);
    __shared__ TcF32BackwardSync sy;
    if (*a.odd) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ktiles = (a.S + kTcRows - 1) / kTcRows;
    long long id = blockIdx.x;
    const int kt = (int)(id % ktiles);
    id /= ktiles;
    const int n = (int)(id % a.N), b = (int)(id / a.N);
    const int j0 = kt * kTcRows;
    const uint8_t* km = a.key_mask ? a.key_mask + b * a.km_sb + n * a.km_sh : nullptr;
    long long first_q = a.causal ? (long long)j0 - (a.S - a.Q) : 0;
    int r0 = first_q <= 0 ? 0 : (int)(first_q < a.Q ? first_q / kTcRows : p.qblocks), r1 = p.qblocks;
    tc_narrow(p, p.ext_k, ktiles, b, n * a.G, a.G, kt, kt, &r0, &r1);
    int nt = a.G * max(0, r1 - r0);
    if (km) {
        const bool any = tid < min(kTcRows, a.S - j0) && km[j0 + tid] != 0;
        if (!__syncthreads_or(any)) nt = 0;
    }
    if (warp == 16) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                tc_bar_init(tc_smem(&sy.full[i]), 1);
                tc_bar_init(tc_smem(&sy.empty[i]), 1);
            }
            tc_bar_init(tc_smem(&sy.own), 1);
            tc_bar_init(tc_smem(&sy.s_full), 1);
            tc_bar_init(tc_smem(&sy.dp_full), 1);
            tc_bar_init(tc_smem(&sy.p_ready), 16);
            tc_bar_init(tc_smem(&sy.ds_ready), 16);
            sy.abort = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    } else if (warp == 17) {
        tmem_alloc(tc_smem(&sy.tmem), 512);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sy.tmem;
    volatile uint32_t* abort = &sy.abort;
    bool ok = true;
    if (warp < 16) {
        // thread = key row, 32 of a tile's 128 queries
        const int w = warp >> 2, wl = warp & 3, row = wl * 32 + lane, j = j0 + row;
        const uint32_t first = lane == 0, lanes = (uint32_t)wl << 21;
        // the warpgroups' sums: dV's channels 0..31, 32..63, dK's
        float sum[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) sum[k] = 0.f;
        const uint32_t sum_at = tmem + (w < 2 ? Cfg::kDV : Cfg::kDK) + (w & 1) * 32 + lanes;
        const int sum_steps = (a.D + 15) / 16 - (w & 1) * 2;
        auto gather = [&]() { add_columns<2>(sum, sum_at, sum_steps); };
        const uint64_t c2 = tc_two(a.c2, a.c2);
        int g = 0, rt = r0;
#pragma unroll 1
        for (int i = 0; i < nt; ++i, rt + 1 < r1 ? ++rt : (++g, rt = r0)) {
            const int q0 = rt * kTcRows + w * 32;
            uint32_t bw = ~0u;
            if (p.bits_t && j < a.S)
                bw = p.bits_t[b * p.bits_t_sb + (n * a.G + g) * p.bits_t_sh + (long long)j * p.Wq + rt * 4 + w];
            if (a.causal) bw &= ~tc_low_bits(j - (a.S - a.Q) - q0);
            const float* l2 = stats + w * 32;
            ok = tc_bar_wait(tc_smem(&sy.full[0]), i & 1, abort, a.err) && tc_bar_wait(tc_smem(&sy.s_full), i & 1, abort, a.err);
            if (!ok) break;
            tc_fence_after();
            float s[32];
            tmem_ld32(reinterpret_cast<uint32_t(&)[32]>(s), tmem + w * 32 + lanes);
            tmem_wait_ld();
            if (__any_sync(0xffffffffu, bw != ~0u)) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    if (!((bw >> k) & 1u)) s[k] = -attn_inf();
            }
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
                const float4 l = *reinterpret_cast<const float4*>(l2 + k);
                tc_split(tc_fma2(tc_two(s[k], s[k + 1]), c2, tc_two(l.x, l.y)), s[k], s[k + 1]);
                tc_split(tc_fma2(tc_two(s[k + 2], s[k + 3]), c2, tc_two(l.z, l.w)), s[k + 2], s[k + 3]);
                s[k] = tc_ex2(s[k]), s[k + 1] = tc_ex2(s[k + 1]), s[k + 2] = tc_ex2(s[k + 2]), s[k + 3] = tc_ex2(s[k + 3]);
            }
            store_pieces_over(tmem, lanes, w, s);
            if (i > 0) {  // the products of the tile before
                ok = tc_bar_wait(tc_smem(&sy.empty[0]), (i - 1) & 1, abort, a.err);
                if (!ok) break;
                tc_fence_after();
                gather();
            }
            tmem_wait_st();
            tc_fence_before();
            tc_bar_arrive_if(first, tc_smem(&sy.p_ready));
            ok = tc_bar_wait(tc_smem(&sy.dp_full), i & 1, abort, a.err);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t d[16];
                tmem_ld16(d, tmem + Cfg::kDP + w * 32 + c * 16 + lanes);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; k += 4) {
                    const float4 l = *reinterpret_cast<const float4*>(l2 + 128 + c * 16 + k);
                    float* x = s + c * 16 + k;
                    tc_split(tc_mul2(tc_add2(tc_two(__uint_as_float(d[k]), __uint_as_float(d[k + 1])), tc_two(l.x, l.y)),
                                     tc_two(x[0], x[1])), x[0], x[1]);
                    tc_split(tc_mul2(tc_add2(tc_two(__uint_as_float(d[k + 2]), __uint_as_float(d[k + 3])), tc_two(l.z, l.w)),
                                     tc_two(x[2], x[3])), x[2], x[3]);
                }
            }
            store_pieces_over(tmem + Cfg::kDP, lanes, w, s);
            tmem_wait_st();
            tc_fence_before();
            tc_bar_arrive_if(first, tc_smem(&sy.ds_ready));
        }
        if (nt > 0 && ok) {
            ok = tc_bar_wait(tc_smem(&sy.empty[0]), (nt - 1) & 1, abort, a.err);
            tc_fence_after();
            if (ok) gather();
        }
        if (ok && j < a.S) {
            const bool live = !km || km[j];
            float* out = static_cast<float*>(w < 2 ? a.dv : a.dk) + (((long long)b * a.S + j) * a.N + n) * a.D;
            store_columns<32>(out, sum, (w & 1) * 32, a.D, w < 2 ? 1.f : a.scale, !live);
        }
    } else {
        const int role = warp - 16;
        if (role == 0 && nt > 0) {
            const uint32_t on = tc_elect(), own = tc_smem(&sy.own);
            tc_bar_expect_if(on, own, 2 * kPieces);
            load_pieces(on, k_tile, &map_k, own, j0, n, b, a.B);
            load_pieces(on, v_tile, &map_v, own, j0, n, b, a.B);
            int g = 0, rt = r0;
            const float* stat = a.row_l2 + ((long long)b * a.M + n * a.G) * p.qblocks * 256;
            for (int i = 0; i < nt; ++i, rt + 1 < r1 ? ++rt : (++g, rt = r0)) {
                const int h = n * a.G + g;
                // dO is let go before Q, and wanted before it
                if (i > 0) ok = tc_bar_wait(tc_smem(&sy.empty[1]), (i - 1) & 1, abort, a.err);
                if (!ok) break;
                tc_bar_expect_if(on, tc_smem(&sy.full[1]), kPieces);
                load_pieces(on, do_tile, &map_do, tc_smem(&sy.full[1]), rt * kTcRows, h, b, a.B);
                if (i > 0) ok = tc_bar_wait(tc_smem(&sy.empty[0]), (i - 1) & 1, abort, a.err);
                if (!ok) break;
                tc_bar_expect_if(on, tc_smem(&sy.full[0]), kPieces + 1024);
                load_pieces(on, q_tile, &map_q, tc_smem(&sy.full[0]), rt * kTcRows, h, b, a.B);
                tc_bulk_if(on, tc_smem(stats), stat + ((long long)g * p.qblocks + rt) * 256, 1024, tc_smem(&sy.full[0]));
            }
        } else if (role == 1 && nt > 0) {
            const uint32_t on = tc_elect();
            const int steps = (a.D + 15) / 16;
            const uint32_t id_s = tc_idesc(true, false, false, 128, 128), id_g = tc_idesc(true, false, true, 128, steps * 16);
            uint32_t step_on[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) step_on[k] = k < steps ? on : 0u;
            const uint64_t k_desc = tc_desc(k_tile, 16, 1024), v_desc = tc_desc(v_tile, 16, 1024);
            const uint64_t q_row = tc_desc(q_tile, 16, 1024), do_row = tc_desc(do_tile, 16, 1024);
            const uint64_t q_col = tc_desc(q_tile, kTcTile, 1024), do_col = tc_desc(do_tile, kTcTile, 1024);
            ok = tc_bar_wait(tc_smem(&sy.own), 0, abort, a.err);
            for (int i = 0; i < nt && ok; ++i) {
                ok = tc_bar_wait(tc_smem(&sy.full[1]), i & 1, abort, a.err);
                if (!ok) break;
                tc_fence_after();
                products_nt(step_on, tmem + Cfg::kDP, v_desc, do_row, id_s);
                tc_commit(on, tc_smem(&sy.dp_full));
                ok = tc_bar_wait(tc_smem(&sy.full[0]), i & 1, abort, a.err);
                if (!ok) break;
                tc_fence_after();
                products_nt(step_on, tmem, k_desc, q_row, id_s);
                tc_commit(on, tc_smem(&sy.s_full));
                ok = tc_bar_wait(tc_smem(&sy.p_ready), i & 1, abort, a.err);
                if (!ok) break;
                tc_fence_after();
                products_tn(on, tmem + Cfg::kDV, tmem, do_col, id_g);
                tc_commit(on, tc_smem(&sy.empty[1]));
                ok = tc_bar_wait(tc_smem(&sy.ds_ready), i & 1, abort, a.err);
                if (!ok) break;
                tc_fence_after();
                products_tn(on, tmem + Cfg::kDK, tmem + Cfg::kDP, q_col, id_g);
                tc_commit(on, tc_smem(&sy.empty[0]));
            }
        }
        __syncwarp();
    }
    if (!ok) tc_drain();
    tc_fence_before();
    __syncthreads();
    if (warp == 17) tmem_dealloc(tmem, 512);
}

struct TcF32Query {
    static constexpr size_t kSmem = 4 * kPieces + 1024;                        // Q, dO, K, V
    static constexpr uint32_t kDP = 128, kDS = 256, kDQ = 448;  // tensor memory: S 0; dS in three pieces of 64
};

__global__ void __launch_bounds__(kF32Threads, 1)
    msda_attention_tc_f32_grad_query_kernel(const TcArgs p, const __grid_constant__ CUtensorMap map_q,
                                            const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                                            const __grid_constant__ CUtensorMap map_do) {
    using Cfg = TcF32Query;
    const AttentionArgs& a = p.a;
    extern __shared__ unsigned char tc_smem_raw[];
    unsigned char* smem = tc_smem_raw + ((1024u - (tc_smem(tc_smem_raw) & 1023u)) & 1023u);
    const uint32_t q_tile = tc_smem(smem), do_tile = q_tile + kPieces, k_tile = q_tile + 2 * kPieces, v_tile = q_tile + 3 * kPieces;
    __shared__ TcF32BackwardSync sy;
    if (*a.odd) return;
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
    if (warp == 16) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                tc_bar_init(tc_smem(&sy.full[i]), 1);
                tc_bar_init(tc_smem(&sy.empty[i]), 1);
            }
            tc_bar_init(tc_smem(&sy.own), 1);
            tc_bar_init(tc_smem(&sy.s_full), 1);
            tc_bar_init(tc_smem(&sy.s_free), 16);
            tc_bar_init(tc_smem(&sy.ds_ready), 16);
            sy.abort = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    } else if (warp == 17) {
        tmem_alloc(tc_smem(&sy.tmem), 512);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sy.tmem;
    volatile uint32_t* abort = &sy.abort;
    bool ok = true;
    if (warp < 16) {
        // thread = query row, 32 of a tile's 128 keys
        const int w = warp >> 2, wl = warp & 3, row = wl * 32 + lane, q = q0 + row;
        const uint32_t first = lane == 0, lanes = (uint32_t)wl << 21;
        const long long r = (((long long)b * a.M + h) * p.qblocks + rt) * 256 + row;
        const float l2 = a.row_l2[r], dl = a.row_dl[r];
        const bool live = l2 != -attn_inf();
        const int seen = live ? tc_seen(a, q) : 0;
        const uint32_t* bits = a.bits && q < a.Q ? a.bits + b * a.bits_sb + h * a.bits_sh + (long long)q * a.W : nullptr;
        const uint64_t c2 = tc_two(a.c2, a.c2), nl = tc_two(l2, l2), nd = tc_two(dl, dl);
        // a warpgroup sums 16 channels
        float sum[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) sum[k] = 0.f;
        const uint32_t sum_at = tmem + Cfg::kDQ + w * 16 + lanes;
        const int sum_steps = (a.D + 15) / 16 - w;
#pragma unroll 1
        for (int i = 0; i < nt; ++i) {
            const int j0 = (t0 + i) * kTcRows + w * 32;
            uint32_t bw = tc_low_bits(seen - j0);
            if (bits) bw &= bits[(t0 + i) * 4 + w];
            if (km) bw &= __ballot_sync(0xffffffffu, j0 + lane < a.S && km[j0 + lane] != 0);
            ok = tc_bar_wait(tc_smem(&sy.s_full), i & 1, abort, a.err);  // dP(i) and dQ(i-1) too
            if (!ok) break;
            tc_fence_after();
            float s[32];
            tmem_ld32(reinterpret_cast<uint32_t(&)[32]>(s), tmem + w * 32 + lanes);
            tmem_wait_ld();
            if (__any_sync(0xffffffffu, bw != ~0u)) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    if (!((bw >> k) & 1u)) s[k] = -attn_inf();
            }
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
                tc_split(tc_fma2(tc_two(s[k], s[k + 1]), c2, nl), s[k], s[k + 1]);
                s[k] = tc_ex2(s[k]), s[k + 1] = tc_ex2(s[k + 1]);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t d[16];
                tmem_ld16(d, tmem + Cfg::kDP + w * 32 + c * 16 + lanes);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                    float* x = s + c * 16 + k;
                    tc_split(tc_mul2(tc_add2(tc_two(__uint_as_float(d[k]), __uint_as_float(d[k + 1])), nd), tc_two(x[0], x[1])), x[0], x[1]);
                }
            }
            tc_fence_before();
            tc_bar_arrive_if(first, tc_smem(&sy.s_free));
            if (i > 0) add_columns<1>(sum, sum_at, sum_steps);
            const uint32_t at = tmem + Cfg::kDS + w * 16 + lanes;
#pragma unroll
            for (int k = 0; k < 2; ++k) store_pieces(s + k * 16, at + k * 8, at + 64 + k * 8, at + 128 + k * 8);
            tmem_wait_st();
            tc_fence_before();
            tc_bar_arrive_if(first, tc_smem(&sy.ds_ready));
        }
        if (nt > 0 && ok) {
            ok = tc_bar_wait(tc_smem(&sy.empty[0]), (nt - 1) & 1, abort, a.err);
            tc_fence_after();
            if (ok) add_columns<1>(sum, sum_at, sum_steps);
        }
        if (ok && q < a.Q) {
            float* out = static_cast<float*>(a.dq) + (((long long)b * a.Q + q) * a.M + h) * a.D;
            store_columns<16>(out, sum, w * 16, a.D, a.scale, !live);
        }
    } else {
        const int role = warp - 16;
        if (role == 0 && nt > 0) {
            const uint32_t on = tc_elect(), own = tc_smem(&sy.own);
            tc_bar_expect_if(on, own, 2 * kPieces);
            load_pieces(on, q_tile, &map_q, own, q0, h, b, a.B);
            load_pieces(on, do_tile, &map_do, own, q0, h, b, a.B);
            for (int i = 0; i < nt; ++i) {  // V is let go behind its scores, K behind dQ
                if (i > 0) ok = tc_bar_wait(tc_smem(&sy.empty[1]), (i - 1) & 1, abort, a.err);
                if (!ok) break;
                tc_bar_expect_if(on, tc_smem(&sy.full[1]), kPieces);
                load_pieces(on, v_tile, &map_v, tc_smem(&sy.full[1]), (t0 + i) * kTcRows, n, b, a.B);
                if (i > 0) ok = tc_bar_wait(tc_smem(&sy.empty[0]), (i - 1) & 1, abort, a.err);
                if (!ok) break;
                tc_bar_expect_if(on, tc_smem(&sy.full[0]), kPieces);
                load_pieces(on, k_tile, &map_k, tc_smem(&sy.full[0]), (t0 + i) * kTcRows, n, b, a.B);
            }
        } else if (role == 1 && nt > 0) {
            const uint32_t on = tc_elect();
            const int steps = (a.D + 15) / 16;
            const uint32_t id_s = tc_idesc(true, false, false, 128, 128), id_g = tc_idesc(true, false, true, 128, steps * 16);
            uint32_t step_on[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) step_on[k] = k < steps ? on : 0u;
            const uint64_t q_desc = tc_desc(q_tile, 16, 1024), do_desc = tc_desc(do_tile, 16, 1024);
            const uint64_t k_row = tc_desc(k_tile, 16, 1024), v_row = tc_desc(v_tile, 16, 1024), k_col = tc_desc(k_tile, kTcTile, 1024);
            auto product_dp = [&](int i) {
                ok = tc_bar_wait(tc_smem(&sy.full[1]), i & 1, abort, a.err);
                if (!ok) return;
                tc_fence_after();
                products_nt(step_on, tmem + Cfg::kDP, do_desc, v_row, id_s);
                tc_commit(on, tc_smem(&sy.empty[1]));
            };
            auto product_s = [&](int i) {
                ok = ok && tc_bar_wait(tc_smem(&sy.full[0]), i & 1, abort, a.err);
                if (!ok) return;
                tc_fence_after();
                products_nt(step_on, tmem, q_desc, k_row, id_s);
                tc_commit(on, tc_smem(&sy.s_full));
            };
            ok = tc_bar_wait(tc_smem(&sy.own), 0, abort, a.err);
            if (ok) product_dp(0);
            product_s(0);
            for (int i = 0; i < nt && ok; ++i) {
                if (i + 1 < nt) {
                    ok = tc_bar_wait(tc_smem(&sy.s_free), i & 1, abort, a.err);
                    if (ok) product_dp(i + 1);
                }
                ok = ok && tc_bar_wait(tc_smem(&sy.ds_ready), i & 1, abort, a.err);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < kPairs; ++e)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        tc_mma_ts(on, tmem + Cfg::kDQ, tmem + Cfg::kDS + kPairA[e] * 64 + k * 8,
                                  k_col + ((kPairB[e] * kTcTile + k * 2048) >> 4), id_g, e > 0 || k > 0);
                tc_commit(on, tc_smem(&sy.empty[0]));
                if (i + 1 < nt) product_s(i + 1);
            }
        }
        __syncwarp();
    }
    if (!ok) tc_drain();
    tc_fence_before();
    __syncthreads();
    if (warp == 17) tmem_dealloc(tmem, 512);
}

// ---- host ----

cudaError_t launch_attention_split(const SplitArgs& a, int tensors, cudaStream_t st) {
    long long most = 1;
    for (int i = 0; i < tensors; ++i) {
        const long long n = ((long long)a.B * a.t[i].rows * a.t[i].heads * (a.Dp / 8) + 255) / 256;
        if (n > most) most = n;
    }
    const dim3 grid((unsigned)(most < kPlanSms * 16 ? most : kPlanSms * 16), (unsigned)tensors);
    msda_attention_split_kernel<<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_attention_tc_f32(const TcArgs& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                    cudaStream_t st) {
    static SmemSeen seen;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(&msda_attention_tc_f32_kernel), TcF32Forward::kSmem, seen);
    if (e != cudaSuccess) return e;
    const long long grid = (long long)p.a.B * p.a.N * p.qblocks * p.a.splits;
    msda_attention_tc_f32_kernel<<<(unsigned)grid, 256, TcF32Forward::kSmem, st>>>(p, q, k, v);
    return cudaGetLastError();
}
cudaError_t launch_attention_tc_f32_grad_key(const TcArgs& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                             const CUtensorMap& g, cudaStream_t st) {
    static SmemSeen seen;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(&msda_attention_tc_f32_grad_key_kernel), TcF32Key::kSmem, seen);
    if (e != cudaSuccess) return e;
    const long long grid = (long long)p.a.B * p.a.N * ((p.a.S + kTcRows - 1) / kTcRows);
    msda_attention_tc_f32_grad_key_kernel<<<(unsigned)grid, kF32Threads, TcF32Key::kSmem, st>>>(p, q, k, v, g);
    return cudaGetLastError();
}
cudaError_t launch_attention_tc_f32_grad_query(const TcArgs& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                               const CUtensorMap& g, cudaStream_t st) {
    static SmemSeen seen;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(&msda_attention_tc_f32_grad_query_kernel), TcF32Query::kSmem, seen);
    if (e != cudaSuccess) return e;
    const long long grid = (long long)p.a.B * p.a.M * p.qblocks;
    msda_attention_tc_f32_grad_query_kernel<<<(unsigned)grid, kF32Threads, TcF32Query::kSmem, st>>>(p, q, k, v, g);
    return cudaGetLastError();
}

}  // namespace msda
