// gdelta_bwd.cu -- the gradients of the gated delta rule in chunks of 64 tokens on the tensor cores (BF16 inputs, r 64 or
// 128, dv 64 or 128).
//
// With the chunk form of gdelta_tc.cu (E = X R, R = V - e^G K S, V' = beta E, Y = scale (e^G Q S + A V'),
// S_next = e^{G_C} S + K^T (e^{G_C - G} V')) and dS the gradient of the state behind the chunk, the chain rule gives
//     D = dL/dV' = scale A^T dY + e^{G_C - G} K dS,      N = dL/dR = X^T (beta D) = dL/dV,
//     dS_before = e^{G_C} dS + Q^T (scale e^G dY) - K^T (e^G N),
// a recurrence over the chunks like the forward one, run backwards.  Then, for every chunk by itself, with dA = scale dY V'^T and
// Z = N E^T, where dec_ij = e^{G_i - G_j}:
//     dP = dA . dec (j <= i),  dL = -Z diag(beta) . dec (j < i)                     gradients of Q K^T and K K^T
//     dQ = dP K + scale e^G dY S^T
//     dK = dP^T Q + dL K + dL^T K - e^G N S^T + beta e^{G_C - G} E dS^T
//     dbeta_j = Z_jj / beta_j                                                       (N_j is beta_j times its error's gradient)
// The gates: dalpha_t = <S_{t-1}, G_t - k_t dv_t^T>, with G_t the gradient of S_t.  Both factors are sums over the chunk's tokens, so
//     alpha_t dalpha_t = sum over j < t <= s of F_sj,     F_sj = dec_sj (P_sj dA_sj - (k_s . k_j) beta_j Z_sj),
// where the state before the chunk stands for a token j = -1 and the gradient behind it for a token s = C:
//     F_s,-1 = e^{G_s} (scale q_s . (dY S^T)_s - k_s . (N S^T)_s),   F_Cj = e^{G_C - G_j} beta_j k_j . (E dS^T)_j,   F_C,-1 = e^{G_C} <S, dS>.
// Every term has alpha_t as a factor, so the division cancels nothing: relative to the two factors' sizes the result is as good at a gate of
// 1e-42 as at 1 (as a difference of the tokens' q . dq and v . dv it was off by 1 % at 1e-3).  Gates below 2^-64 count as that in the
// exponents of F, where it is divided out again, and as 0 in dec elsewhere.
// Kernels: gdelta_prep (A, X, gates, scale e^G Q); the forward chain again, keeping the states between the chunks and E, and beside
// it the backward chain, keeping their gradients and N; and a kernel over all chunks.
// At B4 H16 T4096, 128 wide: 75 us, 241 us (both chains, 128 CTAs; 1.44 GB moved, 6 TB/s) and 254 us (1.14 GB, 4.5 TB/s; 237 before dalpha's
// products with the states went in all parts), so that what the
// kernels hand one another, the states between the chunks and E and N above all, is what bounds them.  Forming each chunk's
// gradients inside the chains would spare half of it, but needs both chains at the same chunk.
// Precision: what reaches an FP32 result (dalpha, dbeta, dS0) takes both BF16 parts of a derived operand (the product of two low
// ones left out); dP and dL, which reach dq and dk only, are rounded to one.

#include "gdelta_tc.cuh"

namespace la {
namespace {

constexpr uint32_t kImg = 128 * 128;             // 16 KB: 128 value columns (rows) x 64 BF16
constexpr uint32_t kTokImg = 2 * kImg;           // E or N: [value column][token], two parts
template <int KD>
constexpr uint32_t kStateImg = KD / 64 * kImg;   // a part of S or dS: [value column][state row] by blocks of 64 rows

// ----------------------------------------------------------------- the chains
// Roles as in gdelta_chain_kernel: the fifth warpgroup brings V to its lanes (forwards) and takes S (dS) of every
// chunk to memory, the sixth takes E (N, and dv).
constexpr int kOwners = 16, kHelpers = 4, kBringer = 16, kTaker = 20, kIssuer = 24, kLoader = 25;
constexpr int kThreads = 896;
constexpr int kGateRing = 4;
constexpr uint32_t kGateStep = 2048;
// registers per thread after the split (launched with 72): 4 x 80 + 48 + 88 + 48 = 7 x 72
constexpr int kRegsOwn = 80, kRegsBring = 48, kRegsTake = 88, kRegsRest = 48;

template <int KD, bool REV>
struct BackCfg {
    static constexpr uint32_t kTK = KD / 64 * kTile;
    // a stage (two): K, V or dY (two blocks of 64 columns), forwards X's parts; backwards one buffer each for X's parts, A's, and
    // scale e^G Q's
    static constexpr uint32_t kSK = 0, kSV = kTK, kSX = kSV + 2 * kTile, kStage = REV ? kSX : kSX + 2 * kTile;
    static constexpr uint32_t kX = 2 * kStage, kA = kX + 2 * kTile, kQ = kA + 2 * kTile, kBufs = REV ? kQ + 2 * kTK : kX;
    // what goes to memory: the state (two parts), and E, or dv (4 KB per warp that takes it)
    static constexpr uint32_t kOutS = kBufs, kOutE = kOutS + 2 * kStateImg<KD>, kGates = kOutE + (REV ? 2 * kTile : kTokImg),
                              kSmall = kGates + kGateRing * kGateStep;
};
// TMEM columns: S^T (two parts), P^T and E^T (then dS^T), (A^T dY)^T, R^T (two parts, then the decayed V'^T's, or the scaled
// N^T's), V^T
constexpr uint32_t kcS = 0, kcP = 128, kcE = 192, kcA = 256, kcR = 320, kcV = 384;

struct alignas(16) BSmall {
    uint64_t full[2], full_x, full_a, full_q;
    uint64_t got_s[2], got_r[2], got_w[2];   // an owner half's operand is in TMEM (8 warps)
    uint64_t got_v, s_read, e_read;          // V^T is there, S has been read (the bringers); E has (the takers)
    uint64_t done0, done1[2], done2[2];      // A^T dY, halves of P, E
    uint64_t done2b;                         // the half of R that comes first has been read
    uint64_t done3[4];                       // halves of dS of even and odd chunks
    uint64_t fin;
    uint32_t tmem_base;
    int abort_flag;
};
#define BBAR(name, i) (sS + (uint32_t)offsetof(BSmall, name) + 8 * (uint32_t)(i))

template <int KD>
constexpr uint32_t kBSmemBytes = (BackCfg<KD, true>::kSmall > BackCfg<KD, false>::kSmall ? BackCfg<KD, true>::kSmall : BackCfg<KD, false>::kSmall) +
                                 sizeof(BSmall) + 1024;
static_assert(kBSmemBytes<128> <= 232448, "shared memory budget");

__device__ __forceinline__ float2 unpack(uint32_t x) { return make_float2(bf16_lo(x), bf16_hi(x)); }

template <int KD, bool REV>
__device__ __forceinline__ void back_chain(const CUtensorMap &map_k, const CUtensorMap &map_v, const GdeltaTcBackArgs &args, int head)
{
    using Cfg = BackCfg<KD, REV>;
    constexpr int KH = KD / 2, KQ = KD / 4;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = align1024(smem_raw);
    BSmall *sm = reinterpret_cast<BSmall *>(base + Cfg::kSmall);
    const uint32_t s0 = smem_u32(base), sS = s0 + Cfg::kSmall;
    auto wait1 = [&](uint32_t bar, uint32_t parity) { return bounded_wait<false>(sS + offsetof(BSmall, abort_flag), bar, parity); };
    auto waitw = [&](uint32_t bar, uint32_t parity) { return bounded_wait<true>(sS + offsetof(BSmall, abort_flag), bar, parity); };

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = args.s.H, dv = args.s.dv, T = args.s.T, nch = (T + kC - 1) / kC;
    const int h = head % H, b = head / H;
    const size_t bh = head;
    auto chunk = [&](int n) { return REV ? nch - 1 - n : n; };

    if (tid == 0) {
        for (uint64_t *bar = sm->full; bar <= &sm->fin; ++bar)
            mbar_init(bar, bar >= sm->got_s && bar < &sm->got_v ? kOwners / 2 : bar >= &sm->got_v && bar <= &sm->e_read ? kHelpers : 1);
        sm->abort_flag = 0;
        fence_mbarrier_init();
    }
    if (warp == kIssuer) {
        tmem_alloc(&sm->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wait_for_last();
    let_next_start();

    if (warp >= kIssuer) {
        regs_dec<kRegsRest>();
        if (warp == kLoader && elect_one()) {
            const int hk = h / (H / args.s.Hk), kh = b * args.s.Hk + hk;
            int n1 = 0, nx = 0, na = 0, nq = 0;        // chunks whose loads were started
#pragma unroll 1
            for (int n = 0; n < nch; ++n) {
                const uint32_t st = s0 + (n & 1) * Cfg::kStage, bar = BBAR(full, n & 1);
                const int c = chunk(n);
                const uint8_t *w = args.ws + (((size_t)b * nch + c) * H + h) * kWsChunkB;
                if (n >= 2 && !wait1(BBAR(done3, 2 + (n & 1)), ((n >> 1) - 1) & 1)) break;
                bar_expect(bar, Cfg::kTK + dv / 64 * kTile + (REV ? 0 : 2 * kTile) + kGateBytesB);
#pragma unroll 1
                for (int x = 0; x < KD / 64; ++x) tma_load(st + Cfg::kSK + x * kTile, &map_k, bar, 64 * x, c * kC, kh);
#pragma unroll 1
                for (int x = 0; x < dv / 64; ++x) tma_load(st + Cfg::kSV + x * kTile, &map_v, bar, 64 * x, c * kC, (int)bh);
                bulk_copy(s0 + Cfg::kGates + (n % kGateRing) * kGateStep, w + kWsGates, kGateBytesB, bar);
                if (!REV) bulk_copy(st + Cfg::kSX, w + kWsX, 2 * kTile, bar);
                n1 = n + 1;
                if (REV) {
                    // one buffer each, as their last reads end
                    if (n > 0 && !wait1(BBAR(done0, 0), (n - 1) & 1)) break;
                    bar_expect(BBAR(full_a, 0), 2 * kTile);
                    bulk_copy(s0 + Cfg::kA, w + kWsA, kTile, BBAR(full_a, 0));
                    bulk_copy(s0 + Cfg::kA + kTile, w + kWsAl, kTile, BBAR(full_a, 0));
                    na = n + 1;
                    if (n > 0 && !wait1(BBAR(done2, 0), (n - 1) & 1)) break;
                    bar_expect(BBAR(full_x, 0), 2 * kTile);
                    bulk_copy(s0 + Cfg::kX, w + kWsX, 2 * kTile, BBAR(full_x, 0));
                    nx = n + 1;
                    if (n > 0 && !wait1(BBAR(done3, 2 + ((n - 1) & 1)), ((n - 1) >> 1) & 1)) break;
                    bar_expect(BBAR(full_q, 0), 2 * Cfg::kTK);
                    bulk_copy(s0 + Cfg::kQ, w + kWsQ, 2 * Cfg::kTK, BBAR(full_q, 0));
                    nq = n + 1;
                }
            }
            // loads still in flight complete before the CTA exits (also after a wait that was given up)
#pragma unroll 1
            for (int i = max(0, n1 - 2); i < n1; ++i) wait1(BBAR(full, i & 1), (i >> 1) & 1);
            if (na) wait1(BBAR(full_a, 0), (na - 1) & 1);
            if (nx) wait1(BBAR(full_x, 0), (nx - 1) & 1);
            if (nq) wait1(BBAR(full_q, 0), (nq - 1) & 1);
        } else if (warp == kIssuer && elect_one()) {
            constexpr uint32_t id64 = idesc_bf16_f32(128, 64, false, false), id32 = idesc_bf16_f32(128, 32, false, REV),
                               idP = idesc_bf16_f32(128, 32, false, false), idS = idesc_bf16_f32(128, KH, false, true),
                               idA = idesc_bf16_f32(128, 64, true, true), idQ = idesc_bf16_f32(128, KH, true, true);
            constexpr uint32_t kHalfRows = (32 * 128) >> 4;
            // (A^T dY)^T = dY^T A, both parts of A
            auto mma_a = [&](int n) {
                const uint32_t st = s0 + (n & 1) * Cfg::kStage;
                const uint32_t ylo = desc_lo(st + Cfg::kSV, kTile), alo = desc_lo(s0 + Cfg::kA, kTile);
#pragma unroll 4
                for (int i = 0; i < 8; ++i) {
                    const uint32_t o = (i & 3) * (2048 >> 4);
                    mma_ss(kcA, ylo + o, kHi128, alo + (i >> 2) * (kTile >> 4) + o, kHi128, idA, i > 0);
                }
                bar_commit(BBAR(done0, 0));
            };
            if (REV && wait1(BBAR(full, 0), 0) && wait1(BBAR(full_a, 0), 0)) {
                tc_fence_after();
                mma_a(0);
            }
#pragma unroll 1
            for (int n = 0; n < nch; ++n) {
                const uint32_t st = s0 + (n & 1) * Cfg::kStage, ph = n & 1;
                const uint32_t klo = desc_lo(st + Cfg::kSK, 16), xlo = desc_lo(REV ? s0 + Cfg::kX : st + Cfg::kSX, REV ? kTile : 16);
                // 1  P^T = S^T K^T
                if (!wait1(BBAR(full, n & 1), (n >> 1) & 1) || !wait1(BBAR(got_s, 0), ph)) break;
                tc_fence_after();
#pragma unroll 4
                for (int i = 0; i < KD / 16; ++i) {
                    const int kk = i >> 1;
                    mma_ts(kcP, kcS + (i & 1) * KH + kk * 8, klo + kk * 2, kHi128, id64, i > 0);
                }
                if (!wait1(BBAR(got_s, 1), ph)) break;
                tc_fence_after();
#pragma unroll 1
                for (int u = 0; u < 2; ++u) {
                    const int t = REV ? 1 - u : u;
                    const uint32_t k2 = klo + t * kHalfRows + ((KD == 128 ? kTile : 64u) >> 4);
#pragma unroll 4
                    for (int i = 0; i < KD / 16; ++i) {
                        const int kk = i >> 1;
                        mma_ts(kcP + 32 * t, kcS + (i & 1) * KH + KD / 4 + kk * 8, k2 + kk * 2, kHi128, idP, true);
                    }
                    bar_commit(BBAR(done1, t));
                }
                // 2  E^T = R^T X^T, the first half of R first; backwards N^T = (beta D)^T X, the second half first
                bool ok = true;
                if (REV && !wait1(BBAR(full_x, 0), ph)) break;
#pragma unroll 1
                for (int u = 0; u < 2; ++u) {
                    const int t = REV ? 1 - u : u;
                    ok = wait1(BBAR(got_r, t), ph);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int w = u; w < 2; ++w) {           // half o of the result from half t of R
                        const int o = REV ? 1 - w : w;
                        const uint32_t d = kcE + 32 * o, r = kcR + 16 * t;
                        // X's rows are the result's tokens forwards, its columns backwards
                        const uint32_t xo = xlo + (REV ? t * kHalfRows + 4 * o : o * kHalfRows + 4 * t);
                        constexpr uint32_t kStep = REV ? 2048 >> 4 : 2;
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk) {
                            mma_ts(d, r + kk * 8, xo + kk * kStep, kHi128, id32, u + kk > 0);
                            mma_ts(d, r + 32 + kk * 8, xo + kk * kStep, kHi128, id32, true);
                            mma_ts(d, r + kk * 8, xo + kk * kStep + (kTile >> 4), kHi128, id32, true);
                        }
                        if (u + w == 0) bar_commit(BBAR(done2, t));
                    }
                    bar_commit(u == 0 ? BBAR(done2b, 0) : BBAR(done2, t));
                }
                if (!ok) break;
                // 3  dS^T = V'^T K; backwards dY^T (scale e^G Q) - (e^G N)^T K.  One half of the state's rows after the other
                // (the second one where E has been read)
                const uint32_t kmn = desc_lo(st + Cfg::kSK, kTile);
                auto mma_q = [&](int t) {                  // both parts of the scaled Q
                    const uint32_t ylo = desc_lo(st + Cfg::kSV, kTile),
                                   qmn = desc_lo(s0 + Cfg::kQ, kTile) + t * ((KD == 128 ? kTile : 64u) >> 4);
#pragma unroll 4
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t o = (i & 3) * (2048 >> 4);
                        mma_ss(kcP + 64 * t, ylo + o, kHi128, qmn + (i >> 2) * (Cfg::kTK >> 4) + o, kHi128, idQ, i > 0);
                    }
                };
                if (REV) {
                    if (!wait1(BBAR(full_q, 0), ph)) break;
                    tc_fence_after();
                    mma_q(0);
                }
                if (!wait1(BBAR(got_w, 0), ph) || !wait1(BBAR(got_w, 1), ph)) break;
                tc_fence_after();
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    const uint32_t half = t * ((KD == 128 ? kTile : 64u) >> 4);
                    if (t == 1) {
                        ok = wait1(BBAR(e_read, 0), ph);
                        if (!ok) break;
                        tc_fence_after();
                        if (REV) mma_q(1);
                    }
#pragma unroll 4
                    for (int i = 0; i < 8; ++i)
                        mma_ts(kcP + 64 * t, kcR + (i >> 2) * 32 + (i & 3) * 8, kmn + half + (i & 3) * (2048 >> 4), kHi128, idS, REV || i > 0);
                    bar_commit(BBAR(done3, 2 * t + (n & 1)));
                }
                if (!ok) break;
                if (REV && n + 1 < nch) {
                    if (!wait1(BBAR(full, (n + 1) & 1), ((n + 1) >> 1) & 1) || !wait1(BBAR(full_a, 0), ph ^ 1)) break;
                    tc_fence_after();
                    mma_a(n + 1);
                }
            }
            // every MMA completes before the CTA exits
            bar_commit(BBAR(fin, 0));
            wait1(BBAR(fin, 0), 0);
        }
        __syncwarp();
    } else if (warp >= kTaker) {
        regs_inc<kRegsTake>();
        const int q4 = warp & 3, d = 32 * q4 + lane;
        const uint32_t tq = (uint32_t)(32 * q4) << 16, buf = s0 + Cfg::kOutE + 4096 * q4;
        const int out_col = 32 * q4 + 8 * (lane & 3), out_tok = lane >> 2;
        const bool first = tid == 32 * kTaker;
        // (a warp that gave up waiting still meets the others at their barriers)
        bool ok = true;
#pragma unroll 1
        for (int n = 0; n < nch; ++n) {
            const int c = chunk(n);
            const uint32_t gates = s0 + Cfg::kGates + (n % kGateRing) * kGateStep;
            uint8_t *img = (REV ? args.N : args.E) + (bh * nch + c) * kTokImg;
            if (!REV) {
                // (the last chunk's E has left its place)
                if (first) tma_store_wait_read<0>();
                named_barrier_sync(1, 32 * kHelpers);
            }
            // E, or N (the gates have been waited for by those whose products this waits for)
            if (ok) ok = waitw(BBAR(done2, 0), n & 1) && waitw(BBAR(done2, 1), n & 1);
            if (ok) {
                tc_fence_after();
                // (all of it at once: the issuer waits for its columns)
                float e4[4][16];
#pragma unroll
                for (int x = 0; x < 4; ++x) tc_ld_32x32b_x16(tq + kcE + 16 * x, e4[x]);
#pragma unroll
                for (int x = 0; x < 4; ++x) wait_loaded(e4[x]);
                tc_fence_before();
                bar_arrive_warp(BBAR(e_read, 0));
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float (&e)[16] = e4[x];
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) split(make_float2(e[2 * i], e[2 * i + 1]), hi[i], lo[i]);
                    if (!REV) {
                        const uint32_t o = s0 + Cfg::kOutE + sw128_offset(d, 2 * x), o2 = s0 + Cfg::kOutE + sw128_offset(d, 2 * x + 1);
                        sts4(o, hi[0], hi[1], hi[2], hi[3]);
                        sts4(o2, hi[4], hi[5], hi[6], hi[7]);
                        sts4(o + kImg, lo[0], lo[1], lo[2], lo[3]);
                        sts4(o2 + kImg, lo[4], lo[5], lo[6], lo[7]);
                    } else {
                        // (there is no room left for N in shared memory: it goes straight to its image)
                        st_row16(img, d, x, hi);
                        st_row16(img + kImg, d, x, lo);
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 g = lds_f4(gates + kGateRatio + 64 * x + 16 * i);
                            w[2 * i] = pack_bf16x2(g.x * e[4 * i], g.y * e[4 * i + 1]);
                            w[2 * i + 1] = pack_bf16x2(g.z * e[4 * i + 2], g.w * e[4 * i + 3]);
                        }
                        cols_put(buf, lane, 2 * x, w[0], w[1], w[2], w[3]);
                        cols_put(buf, lane, 2 * x + 1, w[4], w[5], w[6], w[7]);
                    }
                }
            }
            if (!REV) {
                fence_proxy_async_smem();
                named_barrier_sync(1, 32 * kHelpers);
                if (first && ok) {
                    bulk_store(img, s0 + Cfg::kOutE, kTokImg);
                    tma_store_commit();
                }
            } else if (ok) {
                __syncwarp();
                const int rows = T - c * kC - out_tok;
                uint16_t *y0 = args.dv_out + (bh * T + (size_t)c * kC + out_tok) * dv + out_col;
#pragma unroll 2
                for (int w = 0; w < 8; ++w) {
                    const uint4 v = cols_get(buf, lane, w);
                    if (8 * w < rows && out_col < dv) *reinterpret_cast<uint4 *>(y0 + (size_t)(8 * w) * dv) = v;
                }
                __syncwarp();
            }
        }
        if (!REV && first) tma_store_wait_all<0>();
        tc_fence_before();
    } else if (warp >= kBringer) {
        regs_dec<kRegsBring>();
        const int q4 = warp & 3, d = 32 * q4 + lane;    // lane quadrant, value column
        const uint32_t tq = (uint32_t)(32 * q4) << 16;
        const uint32_t c16 = (d & 63) >> 3, col = (d >> 6) * kTile + (d & 7) * 2;
        const bool live = d < dv;
        const bool first = tid == 32 * kBringer;
        // (a warp that gave up waiting still meets the others at their barriers)
        bool ok = true;
#pragma unroll 1
        for (int n = 0; n < nch; ++n) {
            const int c = chunk(n);
            const uint32_t st = s0 + (n & 1) * Cfg::kStage;
            if (!REV) {
                // V's column (0 past the sequence's end, where TMA fills up), once the last chunk's is used
                if (ok) ok = waitw(BBAR(full, n & 1), (n >> 1) & 1);
                if (ok && n > 0) ok = waitw(BBAR(got_r, 0), (n - 1) & 1) && waitw(BBAR(got_r, 1), (n - 1) & 1);
                if (ok) {
                    tc_fence_after();
#pragma unroll 1
                    for (int x = 0; x < 4; ++x) {
                        uint32_t v[8];
                        const uint32_t a = st + Cfg::kSV + col + x * (16 * 128);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int t = 2 * i;
                            const uint32_t x0 = lds_u16(a + t * 128 + ((c16 ^ (t & 7)) << 4)),
                                           x1 = lds_u16(a + (t + 1) * 128 + ((c16 ^ ((t + 1) & 7)) << 4));
                            v[i] = live ? x0 | x1 << 16 : 0;
                        }
                        tm_st8(tq + kcV + 8 * x, v);
                    }
                    tc_wait_st();
                    tc_fence_before();
                    bar_arrive_warp(BBAR(got_v, 0));
                }
            }
            // the state before the chunk; backwards its gradient behind it, once the last one has left its place
            if (first) tma_store_wait_read<0>();
            named_barrier_sync(2, 32 * kHelpers);
            if (ok) ok = waitw(BBAR(got_s, 0), n & 1) && waitw(BBAR(got_s, 1), n & 1);
            if (ok) {
                tc_fence_after();
#pragma unroll 1
                for (int x = 0; x < KD / 16; ++x) {
                    float hi[8], lo[8];
                    tm_ld8(tq + kcS + 8 * x, hi);
                    tm_ld8(tq + kcS + KH + 8 * x, lo);
                    wait_loaded(hi);
                    wait_loaded(lo);
                    if (x == KD / 16 - 1) {
                        tc_fence_before();
                        bar_arrive_warp(BBAR(s_read, 0));
                    }
                    uint32_t hw[8], lw[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) hw[i] = __float_as_uint(hi[i]), lw[i] = __float_as_uint(lo[i]);
                    const uint32_t o = s0 + Cfg::kOutS + (x >> 2) * kImg + sw128_offset(d, 2 * (x & 3)),
                                   o2 = s0 + Cfg::kOutS + (x >> 2) * kImg + sw128_offset(d, 2 * (x & 3) + 1);
                    sts4(o, hw[0], hw[1], hw[2], hw[3]);
                    sts4(o2, hw[4], hw[5], hw[6], hw[7]);
                    sts4(o + kStateImg<KD>, lw[0], lw[1], lw[2], lw[3]);
                    sts4(o2 + kStateImg<KD>, lw[4], lw[5], lw[6], lw[7]);
                }
                fence_proxy_async_smem();
            }
            named_barrier_sync(2, 32 * kHelpers);
            if (first && ok) {
                bulk_store((REV ? args.dS : args.S) + (bh * nch + c) * (2 * kStateImg<KD>), s0 + Cfg::kOutS,
                           2 * kStateImg<KD>);
                tma_store_commit();
            }
        }
        if (first) tma_store_wait_all<0>();
        tc_fence_before();
    } else {
        regs_inc<kRegsOwn>();
        const int q4 = warp & 3, cq = warp >> 2, ch = cq >> 1, d = 32 * q4 + lane;
        const uint32_t tq = (uint32_t)(32 * q4) << 16;
        const bool live = d < dv;
        const float scale = args.scale;
        const float *S_init = REV ? args.dS_T : args.S0;
        float2 S[KQ / 2];                               // S[i]: state rows KQ cq + 2 i, + 1 of the lane's column
        const size_t s_at = (bh * KD + KQ * cq) * dv + d;
#pragma unroll
        for (int i = 0; i < KQ / 2; ++i) {
            S[i] = make_float2(0.f, 0.f);
            if (S_init && live) S[i] = make_float2(S_init[s_at + (size_t)(2 * i) * dv], S_init[s_at + (size_t)(2 * i + 1) * dv]);
        }
        auto put_s = [&](int x, const float2 *v) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) split(v[i], hi[i], lo[i]);
            tm_st8(tq + kcS + KQ / 2 * cq + 8 * x, hi);
            tm_st8(tq + kcS + KH + KQ / 2 * cq + 8 * x, lo);
        };
        auto stored = [&](uint32_t bar) {
            tc_wait_st();
            tc_fence_before();
            bar_arrive_warp(bar);
        };
#pragma unroll
        for (int x = 0; x < KQ / 16; ++x) put_s(x, S + 8 * x);
        stored(BBAR(got_s, ch));
        bool ok = true;
#pragma unroll 1
        for (int n = 0; n < nch; ++n) {
            const uint32_t ph = n & 1, gates = s0 + Cfg::kGates + (n % kGateRing) * kGateStep + 64 * cq;
            // R^T = V^T - e^G P^T; backwards beta D^T = beta (scale (A^T dY)^T + e^{G_C - G} P^T)
            ok = waitw(BBAR(full, n & 1), (n >> 1) & 1) && waitw(REV ? BBAR(done0, 0) : BBAR(got_v, 0), ph) && waitw(BBAR(done1, ch), ph);
            if (!ok) break;
            tc_fence_after();
            {
                float p[16], v[REV ? 16 : 8];
                tc_ld_32x32b_x16(tq + kcP + 16 * cq, p);
                if constexpr (REV) tc_ld_32x32b_x16(tq + kcA + 16 * cq, v);
                else tm_ld8(tq + kcV + 8 * cq, v);
                wait_loaded(p);
                wait_loaded(v);
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 p0 = make_float2(p[4 * i], p[4 * i + 1]), p1 = make_float2(p[4 * i + 2], p[4 * i + 3]);
                    float2 r0, r1;
                    if constexpr (REV) {
                        const float4 er = lds_f4(gates + 4 * kC + 16 * i), be = lds_f4(gates + 8 * kC + 16 * i);
                        const float2 sc = make_float2(scale, scale);
                        r0 = __fmul2_rn(make_float2(be.x, be.y), __ffma2_rn(sc, make_float2(v[4 * i], v[4 * i + 1]), __fmul2_rn(make_float2(er.x, er.y), p0)));
                        r1 = __fmul2_rn(make_float2(be.z, be.w), __ffma2_rn(sc, make_float2(v[4 * i + 2], v[4 * i + 3]), __fmul2_rn(make_float2(er.z, er.w), p1)));
                    } else {
                        const float4 g = lds_f4(gates + 16 * i);
                        r0 = __ffma2_rn(make_float2(-g.x, -g.y), p0, unpack(__float_as_uint(v[2 * i])));
                        r1 = __ffma2_rn(make_float2(-g.z, -g.w), p1, unpack(__float_as_uint(v[2 * i + 1])));
                    }
                    split(r0, hi[2 * i], lo[2 * i]);
                    split(r1, hi[2 * i + 1], lo[2 * i + 1]);
                }
                tm_st8(tq + kcR + 8 * cq, hi);
                tm_st8(tq + kcR + 32 + 8 * cq, lo);
            }
            stored(BBAR(got_r, ch));
            // beta e^{G_C - G} E^T; backwards -e^G N^T
            ok = waitw(BBAR(done2, ch), ph);
            if (!ok) break;
            tc_fence_after();
            {
                float e[16];
                tc_ld_32x32b_x16(tq + kcE + 16 * cq, e);
                wait_loaded(e);
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 g = lds_f4(gates + (REV ? 0 : 4 * kC) + 16 * i);
                    float4 f = make_float4(-1.f, -1.f, -1.f, -1.f);
                    if (!REV) f = lds_f4(gates + 8 * kC + 16 * i);
                    split(__fmul2_rn(make_float2(g.x, g.y), __fmul2_rn(make_float2(f.x, f.y), make_float2(e[4 * i], e[4 * i + 1]))),
                          hi[2 * i], lo[2 * i]);
                    split(__fmul2_rn(make_float2(g.z, g.w), __fmul2_rn(make_float2(f.z, f.w), make_float2(e[4 * i + 2], e[4 * i + 3]))),
                          hi[2 * i + 1], lo[2 * i + 1]);
                }
                // (the other half of E has read R's half that comes first)
                ok = ch != (REV ? 1 : 0) || waitw(BBAR(done2b, 0), ph);
                if (!ok) break;
                tc_fence_after();
                tm_st8(tq + kcR + 8 * cq, hi);
                tm_st8(tq + kcR + 32 + 8 * cq, lo);
            }
            stored(BBAR(got_w, ch));
            const float gC = ldsf(gates - 64 * cq + 4 * (kC - 1));
            // (the bringers have read S of this chunk before it makes room for the next one's)
            ok = waitw(BBAR(done3, 2 * ch + (n & 1)), (n >> 1) & 1) && waitw(BBAR(s_read, 0), ph);
            if (!ok) break;
            tc_fence_after();
            // (the accumulators of the halves are 64 columns apart)
            const uint32_t from = tq + kcP + 64 * ch + KQ * (cq & 1);
#pragma unroll
            for (int x = 0; x < KQ / 16; ++x) {
                float ds[16];
                tc_ld_32x32b_x16(from + 16 * x, ds);
                wait_loaded(ds);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    S[8 * x + i] = __ffma2_rn(make_float2(gC, gC), S[8 * x + i], make_float2(ds[2 * i], ds[2 * i + 1]));
                put_s(x, S + 8 * x);
            }
            stored(BBAR(got_s, ch));
        }
        if (REV && ok && live) {
#pragma unroll
            for (int i = 0; i < KQ / 2; ++i) {
                args.dS0[s_at + (size_t)(2 * i) * dv] = S[i].x;
                args.dS0[s_at + (size_t)(2 * i + 1) * dv] = S[i].y;
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (tid == 0 && sm->abort_flag) atomicExch(args.s.status, kStatusTimeout);
    if (warp == kIssuer) {
        tc_fence_after();
        tmem_dealloc(sm->tmem_base, 512);
    }
}

// Both chains of every head, side by side: neither needs the other's results.
template <int KD>
__global__ void __launch_bounds__(kThreads, 1)
gdelta_back_chain_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                         const __grid_constant__ CUtensorMap map_dy, const __grid_constant__ GdeltaTcBackArgs args)
{
    if (blockIdx.x & 1) back_chain<KD, false>(map_k, map_v, args, blockIdx.x >> 1);
    else back_chain<KD, true>(map_k, map_dy, args, blockIdx.x >> 1);
}

// -------------------------------------------------- the gradients of a chunk
// One CTA per SM walks the chunks of all heads: 8 warps compute (warp w: rows 16 (w % 4) .. of the M = 64 accumulators, half w / 4
// of their columns), one issues the MMAs, one loads.  What a chunk needs fills shared memory, so the next one's operands come into
// each buffer as soon as its last product has read it, under the products, sums and stores that remain.
constexpr int kGComp = 8, kGIssuer = 8, kGLoader = 9, kGThreads = 320;
template <int KD>
struct GradCfg {
    static constexpr uint32_t kTK = KD / 64 * kTile;
    // Q, K, dY, E's high part and (two buffers, in turn) its low one, N (two parts), S (two parts; then dS's low and high one in
    // their place), dP, dL, the gates (two)
    static constexpr uint32_t kQ = 0, kK = kTK, kY = 2 * kTK, kE = kY + 2 * kTile, kEl = kE + kImg, kN = kEl + 2 * kImg, kS = kN + kTokImg,
                              kP = kS + 2 * kStateImg<KD>, kL = kP + kTile, kGates = kL + kTile,
                              kSmall = kGates + 2 * kGateStep;
};
// TMEM columns: Q K^T, dY E^T, N E^T, K K^T (then dP K and dP^T Q + dL K + dL^T K), dY S^T (then E dS^T), N S^T
constexpr uint32_t kgP = 0, kgYE = 64, kgNE = 128, kgKK = 192, kgQ = 0, kgK = 128, kgYS = 256, kgNS = 384;
struct alignas(16) GSmall {
    uint64_t full[3];              // Q, K, dY, E, N; S; dS
    uint64_t got_p, got_x, got_e;  // dP and dL are in shared memory; dY S^T and S have been read; all accumulators have
    uint64_t doneG, doneS, doneQ, doneF;
    uint64_t fin;
    uint32_t tmem_base;
    int abort_flag;
    // of even and odd chunks (the first warp sums one chunk's up while the others are at the next)
    struct {
        // F over the chunk's own tokens, by blocks of 16 columns: every row's sum; per 16 rows s, for every column t, the sum of
        // F_sj over s >= t and the block's j < t.  F_s,-1 and F_Cj by halves of the state's rows.
        float row[4][kC], part[4][kC], head[2][kC], tail[2][kC];
        float diag[kC], anchor[kGComp];
    } sums[2];
};
#define GBAR(name, i) (sS + (uint32_t)offsetof(GSmall, name) + 8 * (uint32_t)(i))
template <int KD>
constexpr uint32_t kGSmemBytes = GradCfg<KD>::kSmall + sizeof(GSmall) + 1024;
static_assert(kGSmemBytes<128> <= 232448, "shared memory budget");

template <int KD, bool OUT32>
__global__ void __launch_bounds__(kGThreads, 1)
gdelta_grad_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_dy, const __grid_constant__ GdeltaTcBackArgs args, int total)
{
    using Cfg = GradCfg<KD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = align1024(smem_raw);
    GSmall *sm = reinterpret_cast<GSmall *>(base + Cfg::kSmall);
    const uint32_t s0 = smem_u32(base), sS = s0 + Cfg::kSmall;
    auto wait1 = [&](uint32_t bar, uint32_t parity) { return bounded_wait<false>(sS + offsetof(GSmall, abort_flag), bar, parity); };
    auto waitw = [&](uint32_t bar, uint32_t parity) { return bounded_wait<true>(sS + offsetof(GSmall, abort_flag), bar, parity); };

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = args.s.H, dv = args.s.dv, T = args.s.T, nch = (T + kC - 1) / kC;
    const int nit = (total - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;   // chunks of this CTA
    // the i-th: neighbours in time run at the same time, and share the states between them
    auto item = [&](int i) { return (int)blockIdx.x + i * (int)gridDim.x; };

    if (tid == 0) {
        for (uint64_t *bar = sm->full; bar <= &sm->fin; ++bar) mbar_init(bar, bar >= &sm->got_p && bar <= &sm->got_e ? kGComp : 1);
        sm->abort_flag = 0;
        fence_mbarrier_init();
    }
    if (warp == kGIssuer) {
        tmem_alloc(&sm->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wait_for_last();
    let_next_start();

    if (warp == kGLoader) {
        if (elect_one()) {
            bool started = false;        // loads that no wait below has seen land
#pragma unroll 1
            for (int i = 0; i <= nit; ++i) {
                // the i-th chunk's operands, and in between dS of the one before it
                const bool load = i < nit;
                const uint32_t ph = (i - 1) & 1;
                const int g = load ? item(i) : 0, c = g % nch;
                const size_t bh = g / nch;
                const int h = (int)(bh % H), b = (int)(bh / H), kh = b * args.s.Hk + h / (H / args.s.Hk);
                const uint8_t *w = args.ws + (((size_t)b * nch + c) * H + h) * kWsChunkB;
                const uint8_t *E = args.E + (bh * nch + c) * kTokImg, *N = args.N + (bh * nch + c) * kTokImg,
                              *S = args.S + (bh * nch + c) * (2 * kStateImg<KD>);
                const uint32_t f0 = GBAR(full, 0), f1 = GBAR(full, 1);
                if (i > 0 && !wait1(GBAR(got_x, 0), ph)) break;
                if (load) {
                    bar_expect(f0, 2 * Cfg::kTK + dv / 64 * kTile + 2 * kTokImg + kGateBytesB);
                    bar_expect(f1, 2 * kStateImg<KD>);
                    started = true;
                }
                if (i > 0) {
                    const uint8_t *dS = args.dS + (size_t)item(i - 1) * (2 * kStateImg<KD>);
                    bar_expect(GBAR(full, 2), 2 * kStateImg<KD>);
                    bulk_copy(s0 + Cfg::kS + kStateImg<KD>, dS, kStateImg<KD>, GBAR(full, 2));
                    bulk_copy(s0 + Cfg::kS, dS + kStateImg<KD>, kStateImg<KD>, GBAR(full, 2));
                }
                if (load) {
                    bulk_copy(s0 + Cfg::kGates + (i & 1) * kGateStep, w + kWsGates, kGateBytesB, f0);
#pragma unroll 1
                    for (int x = 0; x < dv / 64; ++x) tma_load(s0 + Cfg::kY + x * kTile, &map_dy, f0, 64 * x, c * kC, (int)bh);
                    bulk_copy(s0 + Cfg::kEl + (i & 1) * kImg, E + kImg, kImg, f0);
                    bulk_copy(s0 + Cfg::kN, N, kTokImg, f0);
                    // what has to wait for its buffer comes into L2 meanwhile
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(E), "r"(kImg) : "memory");
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(S), "r"(2 * kStateImg<KD>) : "memory");
                }
                if (i > 0 && !wait1(GBAR(doneQ, 0), ph)) break;
                if (load) {
#pragma unroll 1
                    for (int x = 0; x < KD / 64; ++x) {
                        tma_load(s0 + Cfg::kQ + x * kTile, &map_q, f0, 64 * x, c * kC, kh);
                        tma_load(s0 + Cfg::kK + x * kTile, &map_k, f0, 64 * x, c * kC, kh);
                    }
                }
                if (i > 0 && !wait1(GBAR(doneF, 0), ph)) break;
                if (load) {
                    bulk_copy(s0 + Cfg::kE, E, kImg, f0);
                    bulk_copy(s0 + Cfg::kS, S, 2 * kStateImg<KD>, f1);
                    // (a last chunk's loads have landed when its products are done)
                    started = false;
                }
                if (i == nit) started = false;
            }
            // after a wait that was given up: what was started lands before the CTA exits, or has had the time to
            if (started) wait1(GBAR(full, 0), 0), wait1(GBAR(full, 0), 1), wait1(GBAR(full, 2), 1);
        }
        __syncwarp();
    } else if (warp == kGIssuer) {
        if (elect_one()) {
            constexpr uint32_t M = 64;
            const int nk = dv / 16;
            const uint32_t qk = desc_lo(s0 + Cfg::kQ, 16), kk_ = desc_lo(s0 + Cfg::kK, 16), y = desc_lo(s0 + Cfg::kY, 16),
                           e = desc_lo(s0 + Cfg::kE, kImg), nn = desc_lo(s0 + Cfg::kN, kImg), S = desc_lo(s0 + Cfg::kS, kImg);
            constexpr uint32_t kLo = kImg >> 4, kLoS = kStateImg<KD> >> 4, kMn = 2048 >> 4;
            auto kmaj = [&](int k) { return (uint32_t)((k >> 2) * (kTile >> 4) + (k & 3) * 2); };
#pragma unroll 1
            for (int i = 0; i < nit; ++i) {
                const uint32_t ph = i & 1, el = desc_lo(s0 + Cfg::kEl + ph * kImg, kImg);
                if (!wait1(GBAR(full, 0), ph) || (i > 0 && !wait1(GBAR(got_e, 0), ph ^ 1))) break;
                tc_fence_after();
#pragma unroll 2
                for (int k = 0; k < KD / 16; ++k) {
                    mma_ss(kgP, qk + kmaj(k), kHi128, kk_ + kmaj(k), kHi128, idesc_bf16_f32(M, 64, false, false), k > 0);
                    mma_ss(kgKK, kk_ + kmaj(k), kHi128, kk_ + kmaj(k), kHi128, idesc_bf16_f32(M, 64, false, false), k > 0);
                }
#pragma unroll 1
                for (int k = 0; k < nk; ++k) {
                    constexpr uint32_t idK = idesc_bf16_f32(M, 64, false, true), idM = idesc_bf16_f32(M, 64, true, true);
                    const uint32_t o = k * kMn, ok = kmaj(k);
                    mma_ss(kgYE, y + ok, kHi128, e + o, kHi128, idK, k > 0);
                    mma_ss(kgNE, nn + o, kHi128, e + o, kHi128, idM, k > 0);
                    mma_ss(kgYE, y + ok, kHi128, el + o, kHi128, idK, true);
                    mma_ss(kgNE, nn + o, kHi128, el + o, kHi128, idM, true);
                    mma_ss(kgNE, nn + kLo + o, kHi128, e + o, kHi128, idM, true);
                }
                bar_commit(GBAR(doneG, 0));
                if (!wait1(GBAR(full, 1), ph)) break;
                tc_fence_after();
#pragma unroll 2
                for (int k = 0; k < nk; ++k) {
                    constexpr uint32_t idK = idesc_bf16_f32(M, KD, false, true), idM = idesc_bf16_f32(M, KD, true, true);
                    const uint32_t o = k * kMn, ok = kmaj(k);
                    mma_ss(kgYS, y + ok, kHi128, S + o, kHi128, idK, k > 0);
                    mma_ss(kgNS, nn + o, kHi128, S + o, kHi128, idM, k > 0);
                    mma_ss(kgYS, y + ok, kHi128, S + kLoS + o, kHi128, idK, true);
                    mma_ss(kgNS, nn + o, kHi128, S + kLoS + o, kHi128, idM, true);
                    mma_ss(kgNS, nn + kLo + o, kHi128, S + o, kHi128, idM, true);
                }
                bar_commit(GBAR(doneS, 0));
                if (!wait1(GBAR(got_p, 0), ph)) break;
                tc_fence_after();
                {
                    constexpr uint32_t idK = idesc_bf16_f32(M, KD, false, true), idM = idesc_bf16_f32(M, KD, true, true);
                    const uint32_t qm = desc_lo(s0 + Cfg::kQ, kTile), km = desc_lo(s0 + Cfg::kK, kTile), p = desc_lo(s0 + Cfg::kP, 16),
                                   l = desc_lo(s0 + Cfg::kL, 16);
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        mma_ss(kgQ, p + 2 * k, kHi128, km + k * kMn, kHi128, idK, k > 0);          // dP K
                        mma_ss(kgK, p + k * kMn, kHi128, qm + k * kMn, kHi128, idM, k > 0);        // dP^T Q
                        mma_ss(kgK, l + 2 * k, kHi128, km + k * kMn, kHi128, idK, true);           // dL K
                        mma_ss(kgK, l + k * kMn, kHi128, km + k * kMn, kHi128, idM, true);         // dL^T K
                    }
                }
                bar_commit(GBAR(doneQ, 0));
                if (!wait1(GBAR(full, 2), ph)) break;          // (dS was loaded once S had been read)
                tc_fence_after();
                {
                    constexpr uint32_t idM = idesc_bf16_f32(M, KD, true, true);
#pragma unroll 2
                    for (int k = 0; k < nk; ++k) {                 // dS's high part is in the low one's place
                        const uint32_t o = k * kMn;
                        mma_ss(kgYS, e + o, kHi128, S + kLoS + o, kHi128, idM, k > 0);
                        mma_ss(kgYS, e + o, kHi128, S + o, kHi128, idM, true);
                        mma_ss(kgYS, el + o, kHi128, S + kLoS + o, kHi128, idM, true);
                    }
                }
                bar_commit(GBAR(doneF, 0));
            }
            // every MMA completes before the CTA exits
            bar_commit(GBAR(fin, 0));
            wait1(GBAR(fin, 0), 0);
        }
        __syncwarp();
    } else {
        const int q4 = warp & 3, gq = warp >> 2, i = 16 * q4 + (lane & 15), hl = lane >> 4;
        const uint32_t tq = (uint32_t)(32 * q4) << 16;
        const float scale = args.scale;
        bool ok = true;
        // log2 e^G of a token (no gate below kLeastGate), less another's
        auto log_from = [&](uint32_t gates, int i, float Gh, float Gl) {
            return (ldsf(gates + kGateLog + 8 * i) - Gh) + (ldsf(gates + kGateLog + 8 * i + 4) - Gl);
        };
        // (a warp that gave up waiting still meets the others at their barrier)
#pragma unroll 1
        for (int it = 0; it < nit; ++it) {
            const uint32_t ph = it & 1, gates = s0 + Cfg::kGates + (it & 1) * kGateStep;
            const int c = item(it) % nch;
            const size_t bh = item(it) / nch;
            auto &sums = sm->sums[it & 1];
            float x[KD / 4];                 // scale e^G dY S^T: columns KD / 2 gq + 32 p + 16 hl + u
            uint32_t kw[KD / 8];             // K's there
            ok = ok && waitw(GBAR(full, 0), ph) && waitw(GBAR(doneG, 0), ph);
            float eG = 0.f, eR = 0.f, be = 0.f, Gh = 0.f, Gl = 0.f;
            if (ok) {
                tc_fence_after();
                eG = ldsf(gates + 4 * i), eR = ldsf(gates + 4 * kC + 4 * i), be = ldsf(gates + 8 * kC + 4 * i);
                Gh = ldsf(gates + kGateLog + 8 * i), Gl = ldsf(gates + kGateLog + 8 * i + 4);
                const float closed = ldsf(gates + kGateClosed + 4 * i);
                float P[16], YE[16], NE[16], F[16];
                tc_ld_16x32bx2_x16<16>(tq + kgP + 32 * gq, P);
                tc_ld_16x32bx2_x16<16>(tq + kgYE + 32 * gq, YE);
                tc_ld_16x32bx2_x16<16>(tq + kgNE + 32 * gq, NE);
                tc_ld_16x32bx2_x16<16>(tq + kgKK + 32 * gq, F);
                wait_loaded(P);
                wait_loaded(YE);
                wait_loaded(NE);
                wait_loaded(F);
                const int j0 = 32 * gq + 16 * hl;
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                    const int j = j0 + u;
                    const float bj = ldsf(gates + 8 * kC + 4 * j);
                    const float dec = ex2(-log_from(gates, j, Gh, Gl));
                    const bool open = closed == ldsf(gates + kGateClosed + 4 * j);      // (no gate of about 0 in between)
                    const float dA = scale * bj * YE[u], L = -bj * NE[u];
                    if (j == i) sums.diag[i] = NE[u];
                    F[u] = j < i ? dec * fmaf(P[u], dA, F[u] * L) : 0.f;
                    P[u] = j <= i && open ? dec * dA : 0.f;
                    NE[u] = j < i && open ? dec * L : 0.f;
                }
                const uint32_t o = s0 + sw128_offset(i, j0 >> 3), o2 = s0 + sw128_offset(i, (j0 >> 3) + 1);
                const uint4 p0 = pack8(P), p1 = pack8(P + 8), l0 = pack8(NE), l1 = pack8(NE + 8);
                sts4(o + Cfg::kP, p0.x, p0.y, p0.z, p0.w);
                sts4(o2 + Cfg::kP, p1.x, p1.y, p1.z, p1.w);
                sts4(o + Cfg::kL, l0.x, l0.y, l0.z, l0.w);
                sts4(o2 + Cfg::kL, l1.x, l1.y, l1.z, l1.w);
                fence_proxy_async_smem();
                tc_fence_before();
                bar_arrive_warp(GBAR(got_p, 0));
                // F over the columns before each one of its block, over the rows from that one on: summed over the 16 lanes of the
                // rows, lane l ends with column l
                float run = 0.f;
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                    const float f = F[u];
                    F[u] = j0 + u <= i ? run : 0.f;
                    run += f;
                }
                sums.row[2 * gq + hl][i] = run;
#pragma unroll
                for (int w = 8; w; w >>= 1) {
                    const bool up = lane & w;
#pragma unroll
                    for (int z = 0; z < w; ++z) {
                        const float keep = up ? F[z + w] : F[z], give = up ? F[z] : F[z + w];
                        F[z] = keep + __shfl_xor_sync(0xffffffffu, give, w);
                    }
                }
                sums.part[q4][j0 + (lane & 15)] = F[0];
            }
            ok = ok && waitw(GBAR(full, 1), ph);
            if (ok) {
                // <S, dS>: both are images of the same layout, so any order does
                const uint4 *ds = reinterpret_cast<const uint4 *>(args.dS + (bh * nch + c) * (2 * kStateImg<KD>));
                constexpr int kWords = kStateImg<KD> / 16, kRow = KD / 64 * 8;    // (rows behind dv hold nothing)
                float2 dot = make_float2(0.f, 0.f);
#pragma unroll 4
                for (int y = tid; y < dv * kRow; y += 32 * kGComp) {
                    const int w = y / (dv * 8) * (kImg / 16) + y % (dv * 8);
                    const uint4 dh = ds[w], dl = ds[w + kWords], sh = lds4(s0 + Cfg::kS + 16 * w), sl = lds4(s0 + Cfg::kS + kStateImg<KD> + 16 * w);
                    dot = __ffma2_rn(__fadd2_rn(unpack(dh.x), unpack(dl.x)), __fadd2_rn(unpack(sh.x), unpack(sl.x)), dot);
                    dot = __ffma2_rn(__fadd2_rn(unpack(dh.y), unpack(dl.y)), __fadd2_rn(unpack(sh.y), unpack(sl.y)), dot);
                    dot = __ffma2_rn(__fadd2_rn(unpack(dh.z), unpack(dl.z)), __fadd2_rn(unpack(sh.z), unpack(sl.z)), dot);
                    dot = __ffma2_rn(__fadd2_rn(unpack(dh.w), unpack(dl.w)), __fadd2_rn(unpack(sh.w), unpack(sl.w)), dot);
                }
                float p = dot.x + dot.y;
#pragma unroll
                for (int o = 16; o; o >>= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
                if (lane == 0) sums.anchor[warp] = p;
            }
            ok = ok && waitw(GBAR(doneS, 0), ph);
            if (ok) {
                tc_fence_after();
                const float f = scale * eG;
                float qs = 0.f, ks = 0.f;
#pragma unroll
                for (int p = 0; p < KD / 64; ++p) {
                    const int c0 = KD / 2 * gq + 32 * p;
                    float t[16], ns[16];
                    tc_ld_16x32bx2_x16<16>(tq + kgYS + c0, t);
                    tc_ld_16x32bx2_x16<16>(tq + kgNS + c0, ns);
                    wait_loaded(t);
                    wait_loaded(ns);
                    const int cc = c0 + 16 * hl;
                    const uint32_t qa = s0 + Cfg::kQ + (cc >> 6) * kTile, o0 = sw128_offset(i, (cc & 63) >> 3), o1 = sw128_offset(i, ((cc & 63) >> 3) + 1);
                    const uint4 q0 = lds4(qa + o0), q1 = lds4(qa + o1), k0 = lds4(qa + Cfg::kK + o0), k1 = lds4(qa + Cfg::kK + o1);
                    const uint32_t qw[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w}, kv[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        x[16 * p + 2 * u] = f * t[2 * u];
                        x[16 * p + 2 * u + 1] = f * t[2 * u + 1];
                        qs = fmaf(bf16_lo(qw[u]), t[2 * u], fmaf(bf16_hi(qw[u]), t[2 * u + 1], qs));
                        ks = fmaf(bf16_lo(kv[u]), ns[2 * u], fmaf(bf16_hi(kv[u]), ns[2 * u + 1], ks));
                        kw[8 * p + u] = kv[u];
                    }
                }
                tc_fence_before();
                bar_arrive_warp(GBAR(got_x, 0));
                float head = fmaf(scale, qs, -ks);
                head += __shfl_xor_sync(0xffffffffu, head, 16);
                if (hl == 0) sums.head[gq][i] = ex2(Gh + Gl) * head;
            }
            const int t0 = c * kC;
            ok = ok && waitw(GBAR(doneQ, 0), ph) && waitw(GBAR(doneF, 0), ph);
            if (ok) {
                tc_fence_after();
                const size_t row = (bh * T + t0 + i) * KD;
                const bool in = t0 + i < T;
                const float fe = be * eR;
                float tail = 0.f;
#pragma unroll
                for (int p = 0; p < KD / 64; ++p) {
                    const int c0 = KD / 2 * gq + 32 * p;
                    float a[16], k3[16], ns[16], ed[16];
                    tc_ld_16x32bx2_x16<16>(tq + kgQ + c0, a);
                    tc_ld_16x32bx2_x16<16>(tq + kgK + c0, k3);
                    tc_ld_16x32bx2_x16<16>(tq + kgNS + c0, ns);
                    tc_ld_16x32bx2_x16<16>(tq + kgYS + c0, ed);
                    wait_loaded(a);
                    wait_loaded(k3);
                    wait_loaded(ns);
                    wait_loaded(ed);
                    if (p == KD / 64 - 1) {
                        tc_fence_before();
                        bar_arrive_warp(GBAR(got_e, 0));
                    }
#pragma unroll
                    for (int u = 0; u < 16; ++u) {
                        const uint32_t k2 = kw[8 * p + u / 2];
                        tail = fmaf(u & 1 ? bf16_hi(k2) : bf16_lo(k2), ed[u], tail);
                        a[u] += x[16 * p + u];
                        k3[u] = fmaf(fe, ed[u], fmaf(-eG, ns[u], k3[u]));
                    }
                    if (in) {
                        const size_t at = row + c0 + 16 * hl;
                        if (OUT32) {
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                reinterpret_cast<float4 *>(static_cast<float *>(args.dq) + at)[u] = make_float4(a[4 * u], a[4 * u + 1], a[4 * u + 2], a[4 * u + 3]);
                                reinterpret_cast<float4 *>(static_cast<float *>(args.dk) + at)[u] = make_float4(k3[4 * u], k3[4 * u + 1], k3[4 * u + 2], k3[4 * u + 3]);
                            }
                        } else {
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                reinterpret_cast<uint4 *>(static_cast<uint16_t *>(args.dq) + at)[u] = pack8(a + 8 * u);
                                reinterpret_cast<uint4 *>(static_cast<uint16_t *>(args.dk) + at)[u] = pack8(k3 + 8 * u);
                            }
                        }
                    }
                }
                tail += __shfl_xor_sync(0xffffffffu, tail, 16);
                if (hl == 0) sums.tail[gq][i] = be * ex2(log_from(gates, kC - 1, Gh, Gl)) * tail;
            }
            named_barrier_sync(1, 32 * kGComp);
            if (ok && warp == 0) {
                // alpha_t dalpha_t, two tokens per lane: F over the rows from each one on, of the state before the chunk and of the blocks of
                // columns before the token's own (suffix sums, one per block), of its own block, and of the gradient behind the chunk
                const int a0 = 2 * lane, bt = lane >> 3;
                float h[2], sfx[4], own0 = 0.f, own1 = 0.f, behind = 0.f;
#pragma unroll
                for (int u = 0; u < 2; ++u) h[u] = sums.head[0][a0 + u] + sums.head[1][a0 + u];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (b == bt) own0 = h[0], own1 = h[1];
                    sfx[b] = h[0] + h[1];
#pragma unroll
                    for (int u = 0; u < 2; ++u) h[u] += sums.row[b][a0 + u];
                }
#pragma unroll
                for (int o = 1; o < 32; o <<= 1)
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const float y = __shfl_down_sync(0xffffffffu, sfx[b], o);
                        if (lane + o < 32) sfx[b] += y;
                    }
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const float y = __shfl_down_sync(0xffffffffu, sfx[b], 1);
                    if (b == bt && lane < 31) behind = y;
                }
                const float c0 = sums.tail[0][a0] + sums.tail[1][a0], c1 = sums.tail[0][a0 + 1] + sums.tail[1][a0 + 1];
                float last = c0 + c1;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float y = __shfl_up_sync(0xffffffffu, last, o);
                    if (lane >= o) last += y;
                }
                last = __shfl_up_sync(0xffffffffu, last, 1);
                if (lane == 0) last = 0.f;
                float anchor = 0.f;
                for (int w = 0; w < kGComp; ++w) anchor += sums.anchor[w];
                last = fmaf(ex2(log_from(gates, kC - 1, 0.f, 0.f)), anchor, last);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int t = t0 + a0 + u;
                    if (t >= T) continue;
                    const size_t at = bh * T + t;
                    if (args.dalpha && args.s.alpha) {
                        float d = (u ? behind + own1 : behind + own1 + own0) + (u ? last + c0 : last);
#pragma unroll
                        for (int w = 0; w < 4; ++w) d += sums.part[w][a0 + u];
                        const float al = args.s.alpha[at];
                        args.dalpha[at] = al > 0.f ? d / fmaxf(al, kLeastGate) : 0.f;
                    }
                    if (args.dbeta) args.dbeta[at] = sums.diag[a0 + u] / ldsf(gates + 8 * kC + 4 * (a0 + u));
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (tid == 0 && sm->abort_flag) atomicExch(args.s.status, kStatusTimeout);
    if (warp == kGIssuer) {
        tc_fence_after();
        tmem_dealloc(sm->tmem_base, 512);
    }
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

// The workspace's parts, in order.
struct BackSpace {
    size_t ws, E, N, S, dS, dq, dk, bytes;
};
BackSpace back_space(const GdeltaShape &s)
{
    const size_t heads = (size_t)s.B * s.H, nch = (s.T + kC - 1) / kC, state = (size_t)s.r * 256;
    BackSpace p;
    p.ws = 0;
    p.E = p.ws + heads * nch * kWsChunkB;
    p.N = p.E + heads * nch * kTokImg;
    p.S = p.N + heads * nch * kTokImg;
    p.dS = p.S + heads * nch * 2 * state;
    p.dq = p.dS + heads * nch * 2 * state;
    const size_t part = s.Hk < s.H ? round_up(heads * s.T * s.r * sizeof(float)) : 0;
    p.dk = p.dq + part;
    p.bytes = p.dk + part;
    return p;
}

template <int KD>
cudaError_t launch_as(const GdeltaTcBackMaps &m, GdeltaTcBackArgs a, const GdeltaTcArgs &prep, int sms, cudaStream_t stream)
{
    static OncePerDevice once_c, once_g, once_g32;
    cudaError_t e;
    if ((e = set_smem_once(gdelta_back_chain_kernel<KD>, kBSmemBytes<KD>, once_c)) != cudaSuccess) return e;
    if ((e = set_smem_once(gdelta_grad_kernel<KD, false>, kGSmemBytes<KD>, once_g)) != cudaSuccess) return e;
    if ((e = set_smem_once(gdelta_grad_kernel<KD, true>, kGSmemBytes<KD>, once_g32)) != cudaSuccess) return e;
    const unsigned heads = (unsigned)(a.s.B * a.s.H), chunks = heads * (unsigned)((a.s.T + kC - 1) / kC);
    if ((e = launch_gdelta_prep_backward(m.q, m.k, prep, stream)) != cudaSuccess) return e;
    if ((e = launch_after(gdelta_back_chain_kernel<KD>, 2 * heads, kThreads, kBSmemBytes<KD>, stream, m.k, m.v, m.dy, a)) != cudaSuccess)
        return e;
    const unsigned grid = sms > 0 && (unsigned)sms < chunks ? sms : chunks;
    return launch_after(a.s.Hk < a.s.H ? gdelta_grad_kernel<KD, true> : gdelta_grad_kernel<KD, false>, grid, kGThreads, kGSmemBytes<KD>, stream,
                        m.q, m.k, m.dy, a, (int)chunks);
}

}  // namespace

size_t gdelta_tc_backward_bytes(const GdeltaShape &s) { return back_space(s).bytes; }

cudaError_t launch_gdelta_tc_backward(const GdeltaTcBackMaps &m, const GdeltaShape &s, const GdeltaBackward &g, int sms,
                                      cudaStream_t stream)
{
    const BackSpace p = back_space(s);
    uint8_t *ws = reinterpret_cast<uint8_t *>(g.ws);
    GdeltaTcArgs prep;
    prep.s = s;
    prep.ws = ws + p.ws;
    prep.scale = g.scale;
    GdeltaTcBackArgs a;
    a.s = s;
    a.S0 = g.S0, a.dS_T = g.dS_T, a.dS0 = g.dS0;
    a.dv_out = static_cast<uint16_t *>(g.dv_out);
    a.dalpha = g.dalpha, a.dbeta = g.dbeta;
    a.scale = g.scale;
    a.ws = ws + p.ws, a.E = ws + p.E, a.N = ws + p.N, a.S = ws + p.S, a.dS = ws + p.dS;
    const bool shared = s.Hk < s.H;
    a.dq = shared ? ws + p.dq : g.dq;
    a.dk = shared ? ws + p.dk : g.dk;
    const cudaError_t e = s.r == 64 ? launch_as<64>(m, a, prep, sms, stream) : launch_as<128>(m, a, prep, sms, stream);
    if (e != cudaSuccess || !shared) return e;
    return launch_gdelta_group_sum(s, static_cast<const float *>(a.dq), static_cast<const float *>(a.dk), true, g.dq, g.dk, stream);
}

}  // namespace la
