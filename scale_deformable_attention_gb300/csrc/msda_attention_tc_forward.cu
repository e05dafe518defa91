// msda_attention_tc_forward.cu -- softmax attention on the tensor cores
// (tcgen05, sm_103a), fp16 and bf16, D a multiple of 8 up to 128.
//
//   S = Q K^T,  m = running row maximum,  P = 2^(c S - m),  l += row sums,  O = 2^(m_old - m) O + P V
//
// A block takes NQ tiles of 128 rows of one key head (the G query heads that
// share it lie side by side in a tile, so keys and values are read once for
// all of them) and walks the tiles of 128 keys.  Warps:
//   - one warpgroup a row tile: a thread owns a row, so its maximum and sum need
//     no exchange; it reads S from tensor memory, writes P (16 bits) over it;
//   - one warp issues the TMA copies (a ring of K and V tiles), one a row tile
//     its products, one clears keys that key_mask leaves out.
// With two row tiles the products of one run while the other's exponentials
// are worked out.  O stays in tensor memory.
//
// The reference m is a row's maximum when it was last looked for, not the
// running one: any m that keeps P in range gives the same quotient.  A tile
// takes its exponentials against the m at hand, and only where a row's sum
// then leaves a range (TcForwardRange) are the maximum looked for, O and l
// rescaled and the exponentials taken again.  That is the first tile, and then
// only rows whose scores keep rising; the others save the maximum, which stood
// between reading S and the first exponential (about 500 of 2600 cycles a pair
// of tiles).
//
// bf16 has the range of binary32 and needs the upper limit alone.  f16 has no
// more than 2^-14 with all its bits and 2^-25 at all: m there lies 8 binary
// places below the maximum, so that a P is rounded to half a step or to 2^-33 of
// the row's largest.  That would still lose a row's output where one key
// outweighs the others while its value is small (22222 keys 17.6 below one
// whose value is 0: without the 8 places 0 instead of 5.0e-4 of theirs, with
// them 4e-3 of that off).  Such rows, one key with all but 1/128 of the sum so
// far, have a lower limit too: a tile that falls below it gets an m of its own,
// O and l going up.  Rows whose scores are spread by a standard deviation of 5
// run 17 % longer for both (12: 43 %), others 1 to 2 %, 6 % at 128 channels.
//
// Up to 64 channels P has columns of its own: S(j+1) is made while P(j) is
// still worked out, so a row's warps never wait for a product.  Beyond, P lies
// over S, and S(j+1) is issued behind P(j) V(j) by the same thread: the other
// row tile's exponentials fill that time.
#include "msda_attention_tc.cuh"
#include "msda_attention_tc_host.cuh"
#include "msda_host.cuh"

namespace msda {

// When a row's sum over a tile asks for a new reference m, and where that lies.
// Every P is at most its tile's sum; 128 equal ones at the maximum are 2^15.
template <bool BF16>
struct TcForwardRange {
    static constexpr float kTop = BF16 ? 16384.f : 49152.f;  // the largest sum; f16 holds 65504
    static constexpr float kBelow = BF16 ? 0.f : 8.f;        // m below the maximum
    // f16, rows that one key outweighs: the smallest sum (128 values that add up to it are off by 2^-11 of it at most), m
    // below the maximum when it goes down (room for 2^12 above and 2^10 below), and what keeps O under 2^127: l before, m's way.
    static constexpr float kLow = 0x1p-7f, kBelowLow = 3.f, kMostL = 0x1p40f, kWay = 56.f;
    static constexpr float kAlone = 0x1p-7f;  // of the largest key's P: what the others add up to at most
};

template <int NQ, int NC>
struct TcForwardCfg {
    static constexpr int kStages = NC == 1 ? 8 : 4;  // ring of K and V tiles
    static constexpr int kThreads = NQ * 128 + 128;
    static constexpr uint32_t kTileBytes = NC * kTcTile;
    // tensor memory: S (128 columns a row tile), P (64), O (64 or 128).  With
    // two tiles of up to 128 channels the 512 columns have no room for P: it
    // then lies over S, and the next S waits until P is used up.
    static constexpr bool kOwnP = NC == 1;
    static constexpr uint32_t kP = kOwnP ? NQ * 128 : 0, kPStep = kOwnP ? 64 : 128;
    static constexpr uint32_t kO = kOwnP ? NQ * 192 : NQ * 128;
    static constexpr uint32_t kCols = NQ == 2 ? 512 : 256;
    static constexpr size_t kSmem = (size_t)(NQ + kStages) * kTileBytes + 1024 + 512;
};
// Registers of the two warpgroups on the scores and of the third, 504 together of 3 x 168.  Splits measured within 8 % of one
// another, the best another for each type and width (22223 x 22223, us at 200/104, 208/88, 232/40: f16 at 32 channels
// 1037, 996, 931, at 128 channels 1459, 1504, 1583; bf16 951, 925, 988 and 1452, 1363, 1523).
template <bool BF16, int NC>
struct TcForwardRegs {
    static constexpr int kUp = BF16 ? 208 : NC == 1 ? 232 : 200, kDown = 504 - 2 * kUp;
};

struct TcForwardSync {
    uint64_t full[8], empty[8], ready[8];
    uint64_t q_full, s_full[2], s_free[2], p_full[2], pv_done[2], turn;
    uint32_t tmem, abort;
    uint32_t words[8][4];
};

template <bool BF16, int NQ, int NC>
__global__ void __launch_bounds__(TcForwardCfg<NQ, NC>::kThreads, 1)
    msda_attention_tc_forward_kernel(const TcArgs p, const __grid_constant__ CUtensorMap map_q,
                                     const __grid_constant__ CUtensorMap map_k,
                                     const __grid_constant__ CUtensorMap map_v) {
    using Cfg = TcForwardCfg<NQ, NC>;
    using Range = TcForwardRange<BF16>;
    constexpr int ST = Cfg::kStages;
    const AttentionArgs& a = p.a;
    extern __shared__ unsigned char tc_smem_raw[];
    unsigned char* smem = tc_smem_raw + ((1024u - (tc_smem(tc_smem_raw) & 1023u)) & 1023u);  // stays a shared-memory address to the compiler
    unsigned char* q_tiles = smem;
    unsigned char* ring = smem + NQ * Cfg::kTileBytes;
    __shared__ TcForwardSync sy;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    long long id = blockIdx.x;
    const int split = (int)(id % a.splits);
    id /= a.splits;
    int qb = (int)(id % p.qblocks);
    id /= p.qblocks;
    const int n = (int)(id % a.N), b = (int)(id / a.N);
    if (a.causal) qb = p.qblocks - 1 - qb;  // the rows that see most first
    const int q0 = qb * NQ * p.qpt;         // first query of the block

    // key tiles of this block
    const uint8_t* km = a.key_mask ? a.key_mask + b * a.km_sb + n * a.km_sh : nullptr;
    int t0 = split * a.tiles_per_split;
    int t1 = min(t0 + a.tiles_per_split, (tc_seen(a, min(q0 + NQ * p.qpt, a.Q) - 1) + kTcRows - 1) / kTcRows);
    tc_narrow(p, p.ext_q, (a.Q + kTcRows - 1) / kTcRows, b, n * p.G, p.G, q0 / kTcRows, (min(q0 + NQ * p.qpt, a.Q) - 1) / kTcRows,
              &t0, &t1);
    if (km) tc_trim(km, a.S, &t0, &t1);
    const int nt = max(0, t1 - t0);

    if (warp == NQ * 4) {
        if (lane == 0) {
            for (int i = 0; i < ST; ++i) {
                tc_bar_init(tc_smem(&sy.full[i]), 1);
                tc_bar_init(tc_smem(&sy.empty[i]), NQ);
                tc_bar_init(tc_smem(&sy.ready[i]), 1);
            }
            tc_bar_init(tc_smem(&sy.q_full), 1);
            tc_bar_init(tc_smem(&sy.turn), 1);
            for (int i = 0; i < 2; ++i) {
                tc_bar_init(tc_smem(&sy.s_full[i]), 1);
                tc_bar_init(tc_smem(&sy.s_free[i]), 4);
                tc_bar_init(tc_smem(&sy.p_full[i]), 4);
                tc_bar_init(tc_smem(&sy.pv_done[i]), 1);
            }
            sy.abort = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            tc_prefetch_map(&map_q);
            tc_prefetch_map(&map_k);
            tc_prefetch_map(&map_v);
        }
    } else if (warp == NQ * 4 + 1) {
        tmem_alloc(tc_smem(&sy.tmem), Cfg::kCols);
    }
    if (p.rows < kTcRows) {  // rows that no query fills hold zeros, not what was there
        const uint32_t words = (kTcRows - p.rows) * 8;
        for (uint32_t i = tid; i < NQ * NC * words; i += Cfg::kThreads) {
            const uint32_t c = i / words, w = i - c * words;
            *reinterpret_cast<uint4*>(q_tiles + c * kTcTile + p.rows * 128 + w * 16) = make_uint4(0, 0, 0, 0);
        }
        tc_fence_async();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sy.tmem;
    volatile uint32_t* abort = &sy.abort;

    if (warp < NQ * 4) {
        if constexpr (NQ == 2) tc_regs_up<TcForwardRegs<BF16, NC>::kUp>();
        // ---- softmax: row `row` of tile `t` ----
        const int t = warp >> 2, wl = warp & 3, row = wl * 32 + lane;
        const int q = q0 + t * p.qpt + row / p.G, h = n * p.G + row % p.G;
        const bool valid = row < p.rows && q < a.Q;
        const bool warp_on = __any_sync(0xffffffffu, valid);
        const int seen = valid ? tc_seen(a, q) : 0;
        const int seen_least = __reduce_min_sync(0xffffffffu, valid ? seen : a.S);
        const uint32_t lanes = (uint32_t)wl << 21;  // this warp's lanes of tensor memory
        const uint32_t s_at = tmem + t * 128 + lanes, o_at = tmem + Cfg::kO + t * (NC * 64) + lanes;
        const uint32_t p_at = tmem + Cfg::kP + t * Cfg::kPStep + lanes;
        const uint32_t* bits = a.bits && valid ? a.bits + b * a.bits_sb + h * a.bits_sh + (long long)q * a.W : nullptr;
        const int chunks = (a.D + 15) / 16;
        const uint32_t first = lane == 0;
        // reference, sum; f16: the sum of a tile that asks for a lower reference (0: none), the largest key's part of l
        float m = -attn_inf(), l = 0.f, low = 0.f, alone = 0.f;
#pragma unroll 1
        for (int i = 0; i < nt; ++i) {
            const int j0 = (t0 + i) * kTcRows;
            uint4 bw = make_uint4(~0u, ~0u, ~0u, ~0u);
            if (bits) bw = *reinterpret_cast<const uint4*>(bits + (t0 + i) * 4);
            if (!tc_bar_wait(tc_smem(&sy.s_full[t]), i & 1, abort, a.err)) break;
            tc_fence_after();
            if (warp_on) {
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(s[c], s_at + c * 32);
                tmem_wait_ld();
                if constexpr (Cfg::kOwnP) {  // S(i+1) may be written now
                    tc_fence_before();
                    tc_bar_arrive_if(first, tc_smem(&sy.s_free[t]));
                }
                if (__builtin_expect(km || a.bits || seen_least - j0 < kTcRows, 0)) {
                    const int see = seen - j0;
                    uint32_t w[4] = {bw.x & tc_low_bits(see), bw.y & tc_low_bits(see - 32), bw.z & tc_low_bits(see - 64),
                                     bw.w & tc_low_bits(see - 96)};
                    if (km) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) w[c] &= sy.words[i & 7][c];
                    }
                    if (__builtin_expect(__any_sync(0xffffffffu, (w[0] & w[1] & w[2] & w[3]) != 0xffffffffu), 0)) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!((w[c] >> k) & 1u)) s[c][k] = 0xff800000u;
                    }
                }
                const uint64_t c2 = tc_two(a.c2, a.c2);
                bool gone = false;
                // P = 2^(c S - m) into tensor memory; the row's sum.  `wait`: P(i-1) may still be read.
                auto probabilities = [&](bool wait) {
                    const float ref = m == -attn_inf() ? 0.f : m;
                    const uint64_t nref = tc_two(-ref, -ref);
                    uint64_t part[2] = {0, 0};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            float x0, x1;
                            tc_split(tc_fma2(tc_two(__uint_as_float(s[c][2 * k]), __uint_as_float(s[c][2 * k + 1])), c2, nref), x0,
                                     x1);
                            const float e0 = tc_ex2(x0), e1 = tc_ex2(x1);
                            part[k & 1] = tc_add2(part[k & 1], tc_two(e0, e1));
                            pk[k] = tc_pack<BF16>(e0, e1);
                        }
                        if (c == 0 && wait) {
                            gone = !tc_bar_wait(tc_smem(&sy.pv_done[t]), (i - 1) & 1, abort, a.err);
                            tc_fence_after();
                        }
                        tmem_st16(p_at + c * 16, pk);
                    }
                    float s0, s1;
                    tc_split(tc_add2(part[0], part[1]), s0, s1);
                    return s0 + s1;
                };
                bool renew = __any_sync(0xffffffffu, valid && m == -attn_inf());
                float sum = 0.f;
                if (__builtin_expect(!renew, 1)) {
                    sum = probabilities(Cfg::kOwnP && i > 0);
                    renew = __any_sync(0xffffffffu, valid && !(sum <= Range::kTop && (BF16 || sum >= low)));
                } else if (Cfg::kOwnP && i > 0) {
                    gone = !tc_bar_wait(tc_smem(&sy.pv_done[t]), (i - 1) & 1, abort, a.err);
                    tc_fence_after();
                }
                if (__builtin_expect(renew, 0)) {
                    float mx[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        mx[c] = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
                        for (int k = 2; k < 32; k += 2)
                            mx[c] = tc_max3(mx[c], __uint_as_float(s[c][k]), __uint_as_float(s[c][k + 1]));
                    }
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.c2;
                    float next = fmaxf(m, top - Range::kBelow);
                    if constexpr (!BF16) {
                        if (next > m) alone = exp2f(Range::kBelow);
                        if (low > 0.f && top < m - 6.f && top > m - Range::kWay) next = top - Range::kBelowLow;
                    }
                    const float f = next == m ? 1.f : tc_ex2(m - next);
                    if (!BF16 && next < m) alone *= f;
                    m = next;
                    l *= f;
                    if (i > 0) {
                        for (int c = 0; c < chunks; ++c) {
                            uint32_t o[16];
                            tmem_ld16(o, o_at + c * 16);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tmem_st16(o_at + c * 16, o);
                        }
                    }
                    sum = probabilities(false);
                    if constexpr (!BF16) low = l + sum - alone < alone * Range::kAlone && l < Range::kMostL ? Range::kLow : 0.f;
                }
                if (__builtin_expect(gone, 0)) break;
                l += sum;
                tmem_wait_st();
                tc_fence_before();
            } else if constexpr (Cfg::kOwnP) {
                tc_bar_arrive_if(first, tc_smem(&sy.s_free[t]));
                // a warp without rows may not run a tile ahead of the others: its arrival would count for theirs
                if (i > 0 && !tc_bar_wait(tc_smem(&sy.pv_done[t]), (i - 1) & 1, abort, a.err)) break;
            }
            // the warp's loads and stores of tensor memory have ended for all its lanes (wait::ld and wait::st are
            // instructions of the whole warp): one lane arrives for it
            tc_bar_arrive_if(first, tc_smem(&sy.p_full[t]));
        }
        // ---- output ----
        bool ok = true;
        if (nt > 0) {
            ok = tc_bar_wait(tc_smem(&sy.pv_done[t]), (nt - 1) & 1, abort, a.err);
            tc_fence_after();
        }
        if (warp_on && ok) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const float l2 = l == 0.f ? -attn_inf() : m + log2f(l);
            const long long r = ((long long)b * a.M + h) * a.Q + q;
            const long long part = (long long)split * a.B * a.M * a.Q + r;
            for (int c = 0; c < chunks; ++c) {
                uint32_t o[16];
                if (nt > 0) {
                    tmem_ld16(o, o_at + c * 16);
                    tmem_wait_ld();
                }
                if (!valid) continue;
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = l == 0.f ? 0u : __float_as_uint(__uint_as_float(o[k]) * inv);
                if (a.splits > 1) {
                    float* out = a.part_o + part * a.D + c * 16;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (c * 16 + 4 * k < a.D) reinterpret_cast<uint4*>(out)[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                } else {
                    unsigned char* out = static_cast<unsigned char*>(a.out) +
                                         ((((long long)b * a.Q + q) * a.M + h) * a.D + c * 16) * 2;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = tc_pack<BF16>(__uint_as_float(o[8 * k + 2 * e]), __uint_as_float(o[8 * k + 2 * e + 1]));
                        if (c * 16 + 8 * k < a.D) reinterpret_cast<uint4*>(out)[k] = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
            if (valid) {
                if (a.splits > 1) a.part_lse[part] = l2;
                else a.lse[r] = l2 * kLn2;
            }
        }
        if (!ok) tc_drain();
    } else {
        if constexpr (NQ == 2) tc_regs_down<TcForwardRegs<BF16, NC>::kDown>();
        const int role = warp - NQ * 4;
        bool ok = true;
        if (role == 0 && lane == 0 && nt > 0) {
            // ---- copies ----
            const uint32_t qbar = tc_smem(&sy.q_full);
            tc_bar_expect(qbar, NQ * NC * p.rows * 128);
            for (int t = 0; t < NQ; ++t)
                for (int c = 0; c < NC; ++c)
                    tc_tma_5d(tc_smem(q_tiles) + (t * NC + c) * kTcTile, &map_q, qbar, c * 64, 0, q0 + t * p.qpt, n, b);
            for (int i = 0; i < 2 * nt && ok; ++i) {  // K(0), V(0), K(1), ...
                const int st = i % ST;
                if (i >= ST) ok = tc_bar_wait(tc_smem(&sy.empty[st]), (i / ST - 1) & 1, abort, a.err);
                if (!ok) break;
                const uint32_t bar = tc_smem(&sy.full[st]);
                tc_bar_expect(bar, Cfg::kTileBytes);
                for (int c = 0; c < NC; ++c)
                    tc_tma_5d(tc_smem(ring) + st * Cfg::kTileBytes + c * kTcTile, (i & 1) ? &map_v : &map_k, bar, c * 64, 0,
                              (t0 + (i >> 1)) * kTcRows, n, b);
            }
        } else if ((role == 1 || (NQ == 2 && role == 3)) && nt > 0) {
            // ---- products of row tile t ----
            const int t = role >> 1;
            const uint32_t on = tc_elect();
            const uint32_t id_qk = tc_idesc(BF16, false, false, 128, 128);
            const int steps = (a.D + 15) / 16;
            const uint32_t id_pv = tc_idesc(BF16, false, true, 128, steps * 16);
            uint64_t* full = km ? sy.ready : sy.full;
            const uint32_t ring_at = tc_smem(ring);
            const uint64_t q_desc = tc_desc(tc_smem(q_tiles) + t * Cfg::kTileBytes, 16, 1024);
            const uint32_t s_at = tmem + t * 128, o_at = tmem + Cfg::kO + t * (NC * 64);
            const uint32_t p_at = tmem + Cfg::kP + t * Cfg::kPStep;
            auto product_s = [&](int st) {
                const uint64_t k_desc = tc_desc(ring_at + st * Cfg::kTileBytes, 16, 1024);
#pragma unroll
                for (int k = 0; k < NC * 4; ++k) {  // 16 channels: 32 bytes further, 64: the next tile
                    const uint64_t off = ((k >> 2) * kTcTile + (k & 3) * 32) >> 4;
                    if (k < steps) tc_mma_ss(on, s_at, q_desc + off, k_desc + off, id_qk, k > 0);
                }
                tc_commit(on, tc_smem(&sy.s_full[t]));
            };
            ok = tc_bar_wait(tc_smem(&sy.q_full), 0, abort, a.err) && tc_bar_wait(tc_smem(&full[0]), 0, abort, a.err);
            // P over S: the second row tile starts when the first has worked out its first P, so that from then on
            // the products of one run beside the exponentials of the other (together they took 4200 cycles a pair
            // of tiles of 128 channels)
            if (!Cfg::kOwnP && t == 1) ok = ok && tc_bar_wait(tc_smem(&sy.turn), 0, abort, a.err);
            if (ok) {
                tc_fence_after();
                product_s(0);
                tc_commit(on, tc_smem(&sy.empty[0]));
            }
            for (int i = 0; i < nt && ok; ++i) {
                const int iv = 2 * i + 1, ik = 2 * i + 2;
                const int sv = iv % ST, sk = ik % ST;
                const bool more = i + 1 < nt;
                if (Cfg::kOwnP && more) {
                    ok = tc_bar_wait(tc_smem(&full[sk]), (ik / ST) & 1, abort, a.err) &&
                         tc_bar_wait(tc_smem(&sy.s_free[t]), i & 1, abort, a.err);
                    if (!ok) break;
                    tc_fence_after();
                    product_s(sk);
                    tc_commit(on, tc_smem(&sy.empty[sk]));
                }
                ok = tc_bar_wait(tc_smem(&full[sv]), (iv / ST) & 1, abort, a.err) &&
                     tc_bar_wait(tc_smem(&sy.p_full[t]), i & 1, abort, a.err);
                if (!ok) break;
                tc_fence_after();
                if (!Cfg::kOwnP && NQ == 2 && t == 0 && i == 0) tc_bar_arrive_if(on, tc_smem(&sy.turn));
                const uint64_t v_desc = tc_desc(ring_at + sv * Cfg::kTileBytes, kTcTile, 1024);
#pragma unroll
                for (int k = 0; k < 8; ++k)  // 16 keys: two atoms further
                    tc_mma_ts(on, o_at, p_at + k * 8, v_desc + ((k * 2048) >> 4), id_pv, i > 0 || k > 0);
                tc_commit(on, tc_smem(&sy.pv_done[t]));
                tc_commit(on, tc_smem(&sy.empty[sv]));
                if (!Cfg::kOwnP && more) {
                    ok = tc_bar_wait(tc_smem(&full[sk]), (ik / ST) & 1, abort, a.err);
                    if (!ok) break;
                    tc_fence_after();
                    product_s(sk);
                    tc_commit(on, tc_smem(&sy.empty[sk]));
                }
            }
        } else if (role == 2 && km && nt > 0) {
            // ---- keys that take no part ----
            uint32_t w[4];
            uint8_t next[4];
            auto read = [&](int j0) {
#pragma unroll
                for (int c = 0; c < 4; ++c) next[c] = j0 + c * 32 + lane < a.S ? km[j0 + c * 32 + lane] : 0;
            };
            read(t0 * kTcRows);
            for (int i = 0; i < 2 * nt && ok; ++i) {
                const int st = i % ST;
                if (!(i & 1)) {  // a new tile's keys: their bytes were read a tile ahead
#pragma unroll
                    for (int c = 0; c < 4; ++c) w[c] = __ballot_sync(0xffffffffu, next[c] != 0);
                    if (lane < 4) sy.words[(i >> 1) & 7][lane] = lane == 0 ? w[0] : lane == 1 ? w[1] : lane == 2 ? w[2] : w[3];
                    __syncwarp();
                    if (i + 2 < 2 * nt) read((t0 + (i >> 1) + 1) * kTcRows);
                }
                ok = tc_bar_wait(tc_smem(&sy.full[st]), (i / ST) & 1, abort, a.err);
                if (!ok) break;
                if ((w[0] & w[1] & w[2] & w[3]) != 0xffffffffu) {
                    tc_clear_rows<NC>(ring + st * Cfg::kTileBytes, w, lane);
                    tc_fence_async();
                }
                __syncwarp();
                if (lane == 0) tc_bar_arrive(tc_smem(&sy.ready[st]));
            }
        }
        __syncwarp();
        if (!ok) tc_drain();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == NQ * 4 + 1) tmem_dealloc(tmem, Cfg::kCols);
}

// ---- host ----

template <bool BF16, int NQ, int NC>
static cudaError_t forward_go(const TcArgs& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                              cudaStream_t st) {
    using Cfg = TcForwardCfg<NQ, NC>;
    static SmemSeen seen;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(&msda_attention_tc_forward_kernel<BF16, NQ, NC>), Cfg::kSmem, seen);
    if (e != cudaSuccess) return e;
    const long long grid = (long long)p.a.B * p.a.N * p.qblocks * p.a.splits;
    msda_attention_tc_forward_kernel<BF16, NQ, NC><<<(unsigned)grid, Cfg::kThreads, Cfg::kSmem, st>>>(p, q, k, v);
    return cudaGetLastError();
}

cudaError_t launch_attention_tc_forward(const TcArgs& p, bool bf16, int nq, const CUtensorMap& q, const CUtensorMap& k,
                                        const CUtensorMap& v, cudaStream_t st) {
    const int nc = p.a.D > 64 ? 2 : 1;
#define MSDA_TC_GO(BF, NQ, NC) return forward_go<BF, NQ, NC>(p, q, k, v, st)
    if (bf16) {
        if (nq == 2) {
            if (nc == 1) MSDA_TC_GO(true, 2, 1);
            MSDA_TC_GO(true, 2, 2);
        }
        if (nc == 1) MSDA_TC_GO(true, 1, 1);
        MSDA_TC_GO(true, 1, 2);
    }
    if (nq == 2) {
        if (nc == 1) MSDA_TC_GO(false, 2, 1);
        MSDA_TC_GO(false, 2, 2);
    }
    if (nc == 1) MSDA_TC_GO(false, 1, 1);
    MSDA_TC_GO(false, 1, 2);
#undef MSDA_TC_GO
}

}  // namespace msda
