// gdelta.cu -- the gated delta rule on CUDA cores: the token recurrence in FP32 with its gradients, and
// the single-token step.  (Prompts of the common sizes run in chunks on the tensor cores: gdelta_tc.cu.)
//
// The rule with a gate per token and head:
//     S' = alpha_t S_{t-1},  e_t = v_t - S'^T k_t,  S_t = S' + beta_t k_t e_t^T,  y_t = scale S_t^T q_t.
//
// Its gradients, with G_t = dL/dS_t (what dS_T and the tokens from t on ask of the state):
//     G_t = scale q_t dy_t^T + alpha_{t+1} (G_{t+1} - k_{t+1} dv_{t+1}^T),    G_T = scale q_T dy_T^T + dS_T,
//     lam_t = G_t^T k_t,  dv_t = beta_t lam_t,  dbeta_t = lam_t . e_t,  dS0 = alpha_1 (G_1 - k_1 dv_1^T),
//     dq_t = scale S_t dy_t,   dk_t = beta_t G_t e_t - S'_t dv_t.
// Every column of S is a recurrence of its own given k, and so is every column of G: one sweep forwards
// leaves e, one backwards lam.  With e and dv known every row of S, and of G, is one as well: the products
// S dy, S' dv and G e are two more sweeps over the transposed states.  The gates:
//     dalpha_t = <S_{t-1}, G_t - k_t dv_t^T>,
// formed chunk by chunk from the states that the first two sweeps leave between chunks (gdelta_gate_kernel).

#include "gdelta.h"
#include "launch_after.cuh"
#include "mma_tf32.cuh"
#include "sm103_ptx.cuh"

#include <cuda_bf16.h>
#include <type_traits>

namespace la {
namespace {

template <bool BF16>
__device__ __forceinline__ float load_elem(const void *p, size_t i)
{
    return BF16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16) : static_cast<const float *>(p)[i];
}

template <bool BF16>
__device__ __forceinline__ void store_elem(void *p, size_t i, float x)
{
    if (BF16) static_cast<uint16_t *>(p)[i] = (uint16_t)(pack_bf16x2(x, 0.f) & 0xffffu);
    else static_cast<float *>(p)[i] = x;
}

// ------------------------------------------------------------ the recurrence
// The four sweeps; X is the state (rows x columns), a row vector has an element per row, a column
// element belongs to the lane's column:
//     FWD  X = S    (r x dv), forwards:   X *= alpha;  p = X^T k;  X += k (beta (v - p))^T;  out = scale X^T q;  e = v - p
//     REV  X = G    (r x dv), backwards:  X += q (scale dy)^T;  p = X^T k = lam;  X -= k (beta p)^T;  X *= alpha
//     QUE  X = S^T  (dv x r), forwards:   X *= alpha;  w = X^T dv;  X += e (beta k)^T;  dq = scale X^T dy
//     KEY  X = G^T  (dv x r), backwards:  X += dy (scale q)^T;  m = X^T e;  X -= dv k^T;  X *= alpha;  dk = beta m - w
enum RecMode { kFwd, kRev, kQue, kKey };

struct RecArgs {
    GdeltaShape s;
    const void *q, *k, *v, *dy;
    const float *e, *lam;        // FP32 [B,H,T,dv] (read by kQue, kKey)
    float *e_out, *lam_out;      // (written by kFwd, kRev)
    float *w, *dq;               // FP32 [B,H,T,r]: w of kQue, over which kKey leaves dk; dq
    void *y;                     // kFwd: y or nullptr
    void *dv_out;                // kRev
    const float *S_init;         // [B,H,r,dv] or nullptr
    float *S_fin;                // [B,H,r,dv] or nullptr
    float scale;
    // kFwd in segments of seg_len tokens (nseg > 1): the first pass leaves what each segment adds to the state, N, and what it makes of
    // the one before it, M (S -> M S + N); the second one starts from `starts`
    int nseg = 1, seg_len = 0;
    bool sums = false;
    float *N = nullptr, *M = nullptr;        // [B*H][nseg][r][dv], [B*H][nseg][r][r]
    const float *starts = nullptr;           // [B*H][nseg][r][dv]
    float *ckpt = nullptr;                   // kFwd: the states before every chunk, kRev: the gradients behind it, [B*H][chunks][r][dv]
};

constexpr int kRecTok = 16;              // tokens per staged block
constexpr int kRecComp = 128;            // threads that compute: 4 warps of 8 columns
constexpr int kRecThreads = 2 * kRecComp;   // and as many that stage the next block and write out the last one
constexpr int kRecCols = 32;
constexpr int kRecGroup = 4;             // tokens taken together
constexpr int kGateC = 64;               // tokens per chunk of the gates' gradient
static_assert(kGateC % kRecTok == 0, "chunks end where staged blocks do");

template <int RPL>
constexpr int kRecStageFloats = kRecTok * (3 * 8 * RPL + 4 * kRecCols + 2 + 6);

// Four tokens are taken together, i and j in the sweep's order, X the state before them.  d_j w_j^T is what token j
// writes (d = k, k, e, dv), in the backward sweeps with x_j add_j^T before it; the decays are
//     forwards:   c_i = prod_{l <= i} alpha_l,  m_ji = prod_{j < l <= i} alpha_l;     backwards:  l < i and j <= l < i
//     p_i = c_i X^T b_i + sum_{j < i} m_ji (d_j . b_i) w_j  [+ sum_{j <= i} m_ji (x_j . b_i) add_j, backwards]
//     out_i = c_i X^T x_i + sum_{j <= i} m_ji (d_j . x_i) w_j      (forwards)
// and X takes the four outer products at once.  So only p's chain over four numbers is serial, and the sums over
// the rows are formed side by side.  The ten and six products of the tokens' vectors come from the staging warps.
//
// A warp's lane (g, jj), g = lane / 4, holds rows 4 (8 m + g) + i (m < RPL / 4, i < 4) of the columns 2 jj and
// 2 jj + 1 of its warp's 8; the sums over the rows are exchanged so that group g ends with one of the eight
// (p of token g, or out of token g - 4): 14 shuffles, and 8 to hand p out, where whole sums for all took 48.  The staging
// warps convert a block of 16 tokens to FP32 while the computing ones work on the one before, and store its
// results.  4 r dv FMAs per token and head bound it (FP32 B16 H16 T1001, 128 x 128: 1.0 ms, 33 TFLOP/s of about 75, beside the products
// of the tokens with one another); few heads are bound by a group's latency, 0.4 us at 64 rows (B2 H4 T1001, 64 x 96: 104 us; 240
// token by token, the sums of one waiting for the ones before, and the next block's loads for one another; 84 in segments).
// CKPT: the gradients' first two sweeps with a gate, which leave the state (its gradient) at every chunk's border.
template <int MODE, bool BF16, int RPL, bool CKPT>
__global__ void __launch_bounds__(kRecThreads)
gdelta_rec_kernel(const RecArgs a)
{
    constexpr bool kT = MODE == kQue || MODE == kKey;      // transposed state
    constexpr bool kBack = MODE == kRev || MODE == kKey;
    constexpr int W = 8 * RPL;                             // padded rows
    extern __shared__ __align__(16) float smem[];
    // per stage: row vectors x (q, q, dy, dy), b (k, k, dv, e), d (-, -, e, dv), column elements, results, gates
    float *const st0 = smem;
    constexpr int kOffB = kRecTok * W, kOffD = 2 * kRecTok * W, kOffC = 3 * kRecTok * W, kOffC2 = kOffC + kRecTok * kRecCols,
                  kOffO = kOffC2 + kRecTok * kRecCols, kOffO2 = kOffO + kRecTok * kRecCols, kOffG = kOffO2 + kRecTok * kRecCols,
                  kOffM = kOffG + 2 * kRecTok;      // per group: the products 4 x 4, c, m to the group's end
    constexpr int kStage = kRecStageFloats<RPL>;

    const int tid = threadIdx.x, lane = tid & 31;
    wait_for_last();
    let_next_start();
    const GdeltaShape &s = a.s;
    const bool parts = MODE == kFwd && a.nseg > 1;
    const int b = parts ? blockIdx.z / a.nseg : blockIdx.z, seg = parts ? blockIdx.z % a.nseg : 0, h = blockIdx.y;
    // (M's columns behind N's: the recurrence from the unit matrix, with nothing to write but its own decay)
    const int slices = (s.dv + kRecCols - 1) / kRecCols;
    const bool unit = parts && a.sums && blockIdx.x >= slices;
    const int c0 = (blockIdx.x - (unit ? slices : 0)) * kRecCols;
    const int rows = kT ? s.dv : s.r, cols = kT || unit ? s.r : s.dv;
    const int hk = h / (s.H / s.Hk);
    int T = s.T;
    size_t tok0 = 0;                         // packed: the sequence's first token; in segments: the segment's
    if (parts) {
        tok0 = (size_t)seg * a.seg_len;
        T = min(a.seg_len, s.T - (int)tok0);
    }
    const bool packed = s.cu_seqlens != nullptr;
    if (packed) {
        const int lo = s.cu_seqlens[b], hi = s.cu_seqlens[b + 1];
        if (lo < 0 || hi < lo || hi > s.T) {
            if (tid == 0 && blockIdx.x == 0) atomicExch(s.status, kStatusShape);
            return;
        }
        T = hi - lo;
        tok0 = lo;
    }
    const size_t bh = (size_t)b * s.H + h;
    // element (t, 0) of a token array with `heads` heads, its head hh, d elements a row: first + t * stride
    struct Rows {
        size_t first;
        ptrdiff_t stride;
    };
    auto rows_of = [&](int heads, int hh, int d) -> Rows {
        return packed ? Rows{(tok0 * heads + hh) * (size_t)d, (ptrdiff_t)heads * d} : Rows{(((size_t)b * heads + hh) * s.T + tok0) * d, d};
    };
    const bool computes = tid < kRecComp;
    const int warp = tid >> 5, g = lane >> 2, jl = (warp & 3) * 8 + 2 * (lane & 3);
    const int nblk = (T + kRecTok - 1) / kRecTok;
    // token of position i of block n in the sweep's order.  Blocks are whole 16 tokens of the sequence in both directions: a last one
    // that is not full comes first backwards, behind positions past the sequence's end (zeros, alpha 1).
    auto token = [&](int n, int i) { const int t = n * kRecTok + i; return kBack ? nblk * kRecTok - 1 - t : t; };
    auto staging_sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kRecComp) : "memory"); };
    auto block_sync = [] { asm volatile("bar.sync 2, %0;" ::"n"(kRecThreads) : "memory"); };
    if (!computes) {
        // A staging thread's share of a block: read into registers a block ahead, so that the loads' latency passes
        // while the block before is stored, and not within a block's time.
        constexpr int kRowIters = kRecTok * W / kRecComp, kColIters = kRecTok * kRecCols / kRecComp;
        constexpr int kRowStep = W < kRecComp ? kRecComp / W : 1, kRowParts = W > kRecComp ? W / kRecComp : 1;
        float fx[kRowIters], fb[kRowIters], fd[kT ? kRowIters : 1], fu[kColIters], fu2[MODE == kKey ? kColIters : 1], fal = 1.f, fbe = 1.f;
        const int sid = tid - kRecComp, row0 = sid % W, i_row = sid / W, col = c0 + sid % kRecCols, i_col = sid / kRecCols;
        const Rows key = rows_of(s.Hk, hk, s.r), val = rows_of(s.H, h, s.dv), gate = rows_of(s.H, h, 1), res = rows_of(s.H, h, cols);
        const Rows vec = kT ? val : key, elem = kT ? key : val;
        auto fetch = [&](int n) {
            fal = fbe = 1.f;
            if (sid < kRecTok && token(n, sid) < T) {
                const size_t o = gate.first + token(n, sid) * gate.stride;
                if (s.alpha) fal = s.alpha[o];
                if (s.beta) fbe = s.beta[o];
            }
            size_t o = vec.first + row0 + (ptrdiff_t)token(n, i_row) * vec.stride;
            const ptrdiff_t step = (kBack ? -kRowStep : kRowStep) * vec.stride;
#pragma unroll
            for (int j = 0; j < kRowIters; ++j) {
                const int i = i_row + j / kRowParts * kRowStep, part = j % kRowParts;
                const size_t oj = o + part * kRecComp;
                fx[j] = fb[j] = 0.f;
                if (kT) fd[j] = 0.f;
                if (token(n, i) < T && row0 + part * kRecComp < rows) {
                    fx[j] = load_elem<BF16>(kT ? a.dy : a.q, oj);
                    fb[j] = !kT ? load_elem<BF16>(a.k, oj) : MODE == kQue ? a.lam[oj] : a.e[oj];
                    if (kT) fd[j] = MODE == kQue ? a.e[oj] : a.lam[oj];
                }
                if (part == kRowParts - 1) o += step;
            }
            size_t oc = elem.first + col + (ptrdiff_t)token(n, i_col) * elem.stride;
            const ptrdiff_t cstep = (kBack ? -1 : 1) * (kRecComp / kRecCols) * elem.stride;
#pragma unroll
            for (int j = 0; j < kColIters; ++j) {
                fu[j] = 0.f;
                if (MODE == kKey) fu2[j] = 0.f;
                if (token(n, i_col + j * (kRecComp / kRecCols)) < T && col < cols && !unit) {
                    fu[j] = load_elem<BF16>(kT ? a.k : MODE == kFwd ? a.v : a.dy, oc);
                    if (MODE == kKey) fu2[j] = load_elem<BF16>(a.q, oc);
                }
                oc += cstep;
            }
        };
        auto stage_in = [&](int n) {
            float *st = st0 + (n & 1) * kStage;
            if (sid < kRecTok) st[kOffG + sid] = fal, st[kOffG + kRecTok + sid] = fbe;
            if (kT) staging_sync();
#pragma unroll
            for (int j = 0; j < kRowIters; ++j) {
                const int x = sid + j * kRecComp;
                const float bt = kT ? st[kOffG + kRecTok + x / W] : 1.f;
                st[x] = fx[j];
                st[kOffB + x] = MODE == kQue ? bt * fb[j] : fb[j];
                if (kT) st[kOffD + x] = MODE == kKey ? bt * fd[j] : fd[j];
            }
#pragma unroll
            for (int j = 0; j < kColIters; ++j) {
                st[kOffC + sid + j * kRecComp] = MODE == kRev ? a.scale * fu[j] : fu[j];
                if (MODE == kKey) st[kOffC2 + sid + j * kRecComp] = a.scale * fu2[j];
            }
            staging_sync();
        };
        // One warp: the products of group `gr`, with their decays.  At [i][j], j <= i: d_j . x_i (backwards x_j . b_i); at [j][i], j < i: d_j . b_i
        auto stage_products = [&](int n, int gr) {
            float *st = st0 + (n & 1) * kStage;
            const float *x = st + gr * kRecGroup * W, *b = x + kOffB, *d = kT ? x + kOffD : b;
            float m[16];
#pragma unroll
            for (int z = 0; z < 16; ++z) m[z] = 0.f;
#pragma unroll 2
            for (int row = lane; row < W; row += 32) {
                float xv[4], bv[4], dv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) xv[i] = x[i * W + row], bv[i] = b[i * W + row], dv[i] = kT ? d[i * W + row] : bv[i];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j <= i; ++j) {
                        m[4 * i + j] = kBack ? fmaf(xv[j], bv[i], m[4 * i + j]) : fmaf(dv[j], xv[i], m[4 * i + j]);
                        if (j < i) m[4 * j + i] = fmaf(dv[j], bv[i], m[4 * j + i]);
                    }
            }
#pragma unroll
            for (int w = 8; w; w >>= 1) {        // the lane ends with the sum of m[lane / 2]
                const bool up = lane & (2 * w);
#pragma unroll
                for (int z = 0; z < w; ++z) {
                    const float keep = up ? m[z + w] : m[z], give = up ? m[z] : m[z + w];
                    m[z] = keep + __shfl_xor_sync(0xffffffffu, give, 2 * w);
                }
            }
            m[0] += __shfl_xor_sync(0xffffffffu, m[0], 1);
            float *out = st + kOffM + gr * 24;
            const float *al = st + kOffG + gr * kRecGroup;
            const int z = lane >> 1, i = z >> 2, j = z & 3, lo = min(i, j), hi = max(i, j);
            float dec = 1.f, c = 1.f, end = 1.f;
#pragma unroll
            for (int l = 0; l < 4; ++l) {
                const float av = al[l];
                if (kBack ? l >= lo && l < hi : l > lo && l <= hi) dec *= av;
                if (kBack ? l < lane : l <= lane) c *= av;
                if (kBack ? l >= lane : l > lane) end *= av;
            }
            if (!(lane & 1)) out[z] = dec * m[0];
            if (lane < 4) out[16 + lane] = c, out[20 + lane] = end;
        };
        auto stage_out = [&](int n) {
            const float *st = st0 + (n & 1) * kStage;
            if (col >= cols) return;
            size_t o = res.first + col + (ptrdiff_t)token(n, i_col) * res.stride;
            const ptrdiff_t step = (kBack ? -1 : 1) * (kRecComp / kRecCols) * res.stride;
            float was[kColIters];
#pragma unroll
            for (int j = 0; j < kColIters; ++j)
                if (MODE == kKey && token(n, i_col + j * (kRecComp / kRecCols)) < T) was[j] = a.w[o + j * step];
#pragma unroll
            for (int j = 0; j < kColIters; ++j) {
                const int i = i_col + j * (kRecComp / kRecCols), x = sid + j * kRecComp;
                if (token(n, i) >= T) continue;
                const float out = st[kOffO + x], out2 = st[kOffO2 + x], bt = st[kOffG + kRecTok + i];
                const size_t oj = o + j * step;
                if (MODE == kFwd) {
                    if (a.y) store_elem<BF16>(a.y, oj, a.scale * out);
                    if (a.e_out) a.e_out[oj] = out2;
                } else if (MODE == kRev) {
                    a.lam_out[oj] = out;
                    store_elem<BF16>(a.dv_out, oj, bt * out);
                } else if (MODE == kQue) {
                    a.dq[oj] = a.scale * out;
                    a.w[oj] = out2;
                } else {
                    a.w[oj] = fmaf(bt, out, -was[j]);
                }
            }
        };

        static_assert(kRecTok == kRecGroup * (kRecThreads - kRecComp) / 32, "a group for each staging warp");
        if (nblk > 0) {
            fetch(0);
            stage_in(0);
            stage_products(0, warp - kRecComp / 32);
            if (nblk > 1) fetch(1);
        }
        block_sync();
        for (int n = 0; n < nblk; ++n) {
            if (n > 0) stage_out(n - 1);
            staging_sync();                  // the results are read before their stage is refilled
            if (n + 1 < nblk) {
                stage_in(n + 1);
                stage_products(n + 1, warp - kRecComp / 32);
                if (n + 2 < nblk) fetch(n + 2);
            }
            block_sync();
        }
        if (nblk > 0) stage_out(nblk - 1);
    } else {
        float X[2][RPL];
        const float *S_init = a.S_init ? a.S_init + bh * s.r * s.dv : nullptr;
        if (parts) S_init = a.sums ? nullptr : a.starts + (bh * a.nseg + seg) * s.r * s.dv;
#pragma unroll
        for (int m = 0; m < RPL; ++m) {
            const int row = 4 * (8 * (m >> 2) + g) + (m & 3);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = c0 + jl + c;
                X[c][m] = unit && row == col ? 1.f : 0.f;
                if (S_init && row < rows && col < cols)
                    X[c][m] = S_init[(kT ? (size_t)col * s.dv + row : (size_t)row * s.dv + col)];
            }
        }
        block_sync();
        for (int n = 0; n < nblk; ++n) {
            float *st = st0 + (n & 1) * kStage;
            if constexpr (CKPT) {
                if (kBack ? n == 0 || token(n, 0) % kGateC == kGateC - 1 : token(n, 0) % kGateC == 0) {
                    float *to = a.ckpt + (bh * ((T + kGateC - 1) / kGateC) + token(n, 0) / kGateC) * s.r * s.dv;
#pragma unroll
                    for (int m = 0; m < RPL; ++m) {
                        const int row = 4 * (8 * (m >> 2) + g) + (m & 3);
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            if (row < rows && c0 + jl + c < cols) to[(size_t)row * s.dv + c0 + jl + c] = X[c][m];
                    }
                }
            }
            // groups that hold tokens (those past the sequence's end are zeros, alpha 1)
            const int first = kBack && n == 0 ? (nblk * kRecTok - T) / kRecGroup : 0;
            const int groups = kBack ? kRecTok / kRecGroup : (min(kRecTok, T - n * kRecTok) + kRecGroup - 1) / kRecGroup;
#pragma unroll 1
            for (int gr = first; gr < groups; ++gr) {
                const int i0 = gr * kRecGroup;
                const float4 *xr = reinterpret_cast<const float4 *>(st + i0 * W) + g;
                const float4 *br = reinterpret_cast<const float4 *>(st + kOffB + i0 * W) + g;
                const float4 *dr = kT ? reinterpret_cast<const float4 *>(st + kOffD + i0 * W) + g : br;
                const float4 *mr = reinterpret_cast<const float4 *>(st + kOffM + gr * 24);
                // what the serial part needs, read ahead of it
                const float4 m0 = mr[0], m1 = mr[1], m2 = mr[2], m3 = mr[3], c4 = mr[4], end4 = mr[5];
                const float M[4][4] = {{m0.x, m0.y, m0.z, m0.w}, {m1.x, m1.y, m1.z, m1.w}, {m2.x, m2.y, m2.z, m2.w}, {m3.x, m3.y, m3.z, m3.w}};
                const float cv[4] = {c4.x, c4.y, c4.z, c4.w}, end[4] = {end4.x, end4.y, end4.z, end4.w};
                const float4 be4 = *reinterpret_cast<const float4 *>(st + kOffG + kRecTok + i0);
                const float be[4] = {be4.x, be4.y, be4.z, be4.w};
                float u[4][2], add[4][2], row[4], cg = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 cu = *reinterpret_cast<const float2 *>(st + kOffC + (i0 + i) * kRecCols + jl);
                    float2 ad = cu;
                    if (MODE == kKey) ad = *reinterpret_cast<const float2 *>(st + kOffC2 + (i0 + i) * kRecCols + jl);
                    u[i][0] = cu.x, u[i][1] = cu.y, add[i][0] = ad.x, add[i][1] = ad.y;
                    row[i] = 0.f;
                }
                if (!kBack) {           // the row of out's token
                    const float4 r4 = mr[g & 3];
                    row[0] = r4.x, row[1] = (g & 3) >= 1 ? r4.y : 0.f, row[2] = (g & 3) >= 2 ? r4.z : 0.f, row[3] = (g & 3) == 3 ? r4.w : 0.f;
                    cg = st[kOffM + gr * 24 + 16 + (g & 3)];
                }
                // sums[0..3] X^T b, sums[4..7] X^T x (forwards)
                constexpr int kSums = kBack ? 4 : 8;
                float sums[kSums][2];
#pragma unroll
                for (int i = 0; i < kSums; ++i) sums[i][0] = sums[i][1] = 0.f;
#pragma unroll
                for (int m4 = 0; m4 < RPL / 4; ++m4)
#pragma unroll
                    for (int i = 0; i < kSums; ++i) {
                        const float4 vb = i < 4 ? br[i * (W / 4) + 8 * m4] : xr[(i - 4) * (W / 4) + 8 * m4];
                        const float bb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
                        for (int z = 0; z < 4; ++z)
#pragma unroll
                            for (int c = 0; c < 2; ++c) sums[i][c] = fmaf(X[c][4 * m4 + z], bb[z], sums[i][c]);
                    }
                if (kBack) {            // group g and g + 4 end with the same
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int c = 0; c < 2; ++c) sums[i][c] += __shfl_xor_sync(0xffffffffu, sums[i][c], 16);
                }
#pragma unroll
                for (int w = kSums / 2; w; w >>= 1) {
                    const bool up = g & w;
#pragma unroll
                    for (int i = 0; i < w; ++i)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float keep = up ? sums[i + w][c] : sums[i][c], give = up ? sums[i][c] : sums[i + w][c];
                            sums[i][c] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * w);
                        }
                }
                float p[4][2], w[4][2];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float t = cv[i] * __shfl_sync(0xffffffffu, sums[0][c], 4 * i + (lane & 3));
#pragma unroll
                        for (int j = 0; j <= i; ++j) {
                            if (kBack) t = fmaf(M[i][j], add[j][c], t);
                            if (j < i) t = fmaf(M[j][i], w[j][c], t);
                        }
                        p[i][c] = MODE == kFwd ? u[i][c] - t : t;
                        w[i][c] = MODE == kFwd ? be[i] * p[i][c] : MODE == kRev ? -be[i] * t : MODE == kQue ? be[i] * u[i][c] : -u[i][c];
                    }
                float o[2];             // groups 0 to 3: p of token g; 4 to 7: out of token g - 4
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float p01 = g & 1 ? p[1][c] : p[0][c], p23 = g & 1 ? p[3][c] : p[2][c];
                    o[c] = g & 2 ? p23 : p01;
                    if (!kBack) {
                        float out = cg * sums[0][c];
#pragma unroll
                        for (int j = 0; j < 4; ++j) out = fmaf(row[j], w[j][c], out);
                        o[c] = g & 4 ? out : o[c];
                    }
                }
                if (!kBack || g < 4)
                    *reinterpret_cast<float2 *>(st + (kBack || g >= 4 ? kOffO : kOffO2) + (i0 + (g & 3)) * kRecCols + jl) = make_float2(o[0], o[1]);
                const float all = kBack ? end[0] : cv[3];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c) w[i][c] *= end[i], add[i][c] *= end[i];
#pragma unroll
                for (int m4 = 0; m4 < RPL / 4; ++m4) {
#pragma unroll
                    for (int z = 0; z < 4; ++z)
#pragma unroll
                        for (int c = 0; c < 2; ++c) X[c][4 * m4 + z] *= all;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 vd = dr[i * (W / 4) + 8 * m4];
                        const float dd[4] = {vd.x, vd.y, vd.z, vd.w};
                        const float4 vx = kBack ? xr[i * (W / 4) + 8 * m4] : vd;
                        const float xx[4] = {vx.x, vx.y, vx.z, vx.w};
#pragma unroll
                        for (int z = 0; z < 4; ++z)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                float &X1 = X[c][4 * m4 + z];
                                X1 = fmaf(dd[z], w[i][c], X1);
                                if (kBack) X1 = fmaf(xx[z], add[i][c], X1);
                            }
                    }
                }
            }
            block_sync();
        }
        float *S_fin = a.S_fin ? a.S_fin + bh * s.r * s.dv : nullptr;
        if (parts && a.sums) S_fin = unit ? a.M + (bh * a.nseg + seg) * s.r * s.r : a.N + (bh * a.nseg + seg) * s.r * s.dv;
        else if (parts && seg < a.nseg - 1) S_fin = nullptr;
        const int width = unit ? s.r : s.dv;
        if (S_fin) {
#pragma unroll
            for (int m = 0; m < RPL; ++m) {
                const int row = 4 * (8 * (m >> 2) + g) + (m & 3);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int col = c0 + jl + c;
                    if (row < rows && col < cols)
                        S_fin[kT ? (size_t)col * s.dv + row : (size_t)row * width + col] = X[c][m];
                }
            }
        }
        }
}

template <int MODE, bool BF16, int RPL, bool CKPT = false>
cudaError_t launch_rec_as(const RecArgs &a, cudaStream_t stream)
{
    if constexpr (!CKPT && (MODE == kFwd || MODE == kRev))
        if (a.ckpt) return launch_rec_as<MODE, BF16, RPL, true>(a, stream);
    static OncePerDevice once;
    constexpr uint32_t bytes = 2 * kRecStageFloats<RPL> * 4;
    const cudaError_t e = set_smem_once(gdelta_rec_kernel<MODE, BF16, RPL, CKPT>, bytes, once);
    if (e != cudaSuccess) return e;
    const int cols = MODE == kQue || MODE == kKey ? a.s.r : a.s.dv;
    unsigned slices = (cols + kRecCols - 1) / kRecCols;
    if (a.sums) slices += (a.s.r + kRecCols - 1) / kRecCols;
    const dim3 grid(slices, a.s.H, a.s.B * a.nseg);
    if (a.nseg > 1 && !a.sums) return launch_after(gdelta_rec_kernel<MODE, BF16, RPL, CKPT>, grid, kRecThreads, bytes, stream, a);
    gdelta_rec_kernel<MODE, BF16, RPL, CKPT><<<grid, kRecThreads, bytes, stream>>>(a);
    return cudaGetLastError();
}

template <int MODE>
cudaError_t launch_rec(const RecArgs &a, bool bf16, cudaStream_t stream)
{
    const int rows = MODE == kQue || MODE == kKey ? a.s.dv : a.s.r;
    if (rows <= 64) return bf16 ? launch_rec_as<MODE, true, 8>(a, stream) : launch_rec_as<MODE, false, 8>(a, stream);
    if (rows <= 128) return bf16 ? launch_rec_as<MODE, true, 16>(a, stream) : launch_rec_as<MODE, false, 16>(a, stream);
    return bf16 ? launch_rec_as<MODE, true, 32>(a, stream) : launch_rec_as<MODE, false, 32>(a, stream);
}

// The states before the segments: S <- M S + N from one segment to the next.  A CTA has 32 columns of a head's state in shared memory
// and takes M by 8 RW rows of up to 32 KW columns; a warp forms RW of them, and what comes next is loaded meanwhile.
template <int RW, int KW>
__global__ void __launch_bounds__(256)
gdelta_join_kernel(GdeltaShape s, const float *__restrict__ S0, const float *N, const float *M, float *starts, int nseg)
{
    extern __shared__ __align__(16) float sm_join[];
    const int r = s.r, dv = s.dv, rp = (r + 3) & ~3;        // (columns of M up to rp are 0)
    float *St = sm_join, *Sn = St + rp * 32, *Mt = Sn + rp * 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, col = blockIdx.x * 32 + lane;
    const size_t bh = blockIdx.y;
    const bool live = col < dv;
    wait_for_last();
    let_next_start();
    for (int row = warp; row < rp; row += 8) St[row * 32 + lane] = S0 && live && row < r ? S0[(bh * r + row) * dv + col] : 0.f;
    const int tiles = (r + 8 * RW - 1) / (8 * RW), steps = tiles * (nseg - 1);
    Mt += warp * RW * rp;                                   // a warp's rows are its own
    float next[RW][KW], nn[RW];
    auto fetch = [&](int i) {
        const size_t at = bh * nseg + i / tiles;
        const int row0 = i % tiles * (8 * RW) + RW * warp;
#pragma unroll
        for (int j = 0; j < RW; ++j) {
            const int row = row0 + j;
            const float *Mr = M + (at * r + row) * r;
#pragma unroll
            for (int k = 0; k < KW; ++k) next[j][k] = row < r && lane + 32 * k < r ? Mr[lane + 32 * k] : 0.f;
            nn[j] = live && row < r ? N[(at * r + row) * dv + col] : 0.f;
        }
    };
    auto leave = [&](int seg, const float *from) {
        for (int row = warp; row < r; row += 8)
            if (live) starts[((bh * nseg + seg) * r + row) * dv + col] = from[row * 32 + lane];
    };
    if (steps > 0) fetch(0);
    __syncthreads();
    leave(0, St);
    for (int i = 0; i < steps; ++i) {
        const int row0 = i % tiles * (8 * RW) + RW * warp;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < RW; ++j)
#pragma unroll
            for (int k = 0; k < KW; ++k)
                if (lane + 32 * k < rp) Mt[j * rp + lane + 32 * k] = next[j][k];
        float acc[RW];
#pragma unroll
        for (int j = 0; j < RW; ++j) acc[j] = nn[j];
        __syncwarp();
        if (i + 1 < steps) fetch(i + 1);
#pragma unroll 2
        for (int u = 0; u < rp; u += 4) {
            const float x[4] = {St[u * 32 + lane], St[(u + 1) * 32 + lane], St[(u + 2) * 32 + lane], St[(u + 3) * 32 + lane]};
#pragma unroll
            for (int j = 0; j < RW; ++j) {
                const float4 m = *reinterpret_cast<const float4 *>(Mt + j * rp + u);
                acc[j] = fmaf(m.x, x[0], fmaf(m.y, x[1], fmaf(m.z, x[2], fmaf(m.w, x[3], acc[j]))));
            }
        }
#pragma unroll
        for (int j = 0; j < RW; ++j)
            if (row0 + j < rp) Sn[(row0 + j) * 32 + lane] = acc[j];
        if (i % tiles == tiles - 1) {
            __syncthreads();
            float *x = St;
            St = Sn, Sn = x;
            leave(i / tiles + 1, St);
        }
    }
}

// ------------------------------------------------- the gradients' last passes
__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// dbeta_t = lam . e: one warp per (b, h, t).
__global__ void __launch_bounds__(256)
gdelta_beta_kernel(GdeltaShape s, const float *lam, const float *e, float *dbeta)
{
    const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (i >= (long long)s.B * s.H * s.T) return;
    float db = 0.f;
    for (int x = lane; x < s.dv; x += 32) db = fmaf(lam[i * s.dv + x], e[i * s.dv + x], db);
    db = warp_sum(db);
    if (lane == 0) dbeta[i] = db;
}

// dq and dk of a key head: the sum over the value heads that share it, in their order.
template <bool BF16>
__global__ void __launch_bounds__(256)
gdelta_group_sum_kernel(GdeltaShape s, const float *dq, const float *dk, void *dq_out, void *dk_out)
{
    wait_for_last();
    const long long n = (long long)s.T * s.r, i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= n * s.B * s.Hk) return;
    const int group = s.H / s.Hk;
    const size_t from = (i / n) * group * n + i % n;
    float a = 0.f, c = 0.f;
    for (int u = 0; u < group; ++u) {
        a += dq[from + u * n];
        c += dk[from + u * n];
    }
    store_elem<BF16>(dq_out, i, a);
    store_elem<BF16>(dk_out, i, c);
}

// dalpha_t = <S_{t-1}, G_t - k_t dv_t^T> of a chunk's tokens, one CTA per chunk and head.  With S the state before the chunk, G the
// gradient behind it and v'_j = beta_j e_j, both factors are sums over the chunk's tokens,
//     S_{t-1} = (prod_{l < t} alpha_l) S + sum_{j < t} (prod_{j < l < t} alpha_l) k_j v'_j^T,
//     G_t - k_t dv_t^T = (prod_{l > t} alpha_l) G + sum_{s >= t} (prod_{t < l <= s} alpha_l) (scale q_s dy_s^T - k_s dv_s^T),
// so alpha_t dalpha_t is the sum over j < t <= s of F_sj = (prod_{j < l <= s} alpha_l) W_sj, where
//     W_sj = scale (q_s . k_j) (dy_s . v'_j) - (k_s . k_j) (dv_s . v'_j),
// the state before the chunk stands for a token j = -1 (W_s,-1 = scale q_s . S dy_s - k_s . S dv_s) and the gradient behind it for a token
// s = 64 (W_64,j = k_j . G v'_j, W_64,-1 = <S, G>).  Every term of the sum has alpha_t as a factor: nothing cancels that is larger than the
// result by 1 / alpha_t, as the difference of the tokens' q . dq and v . dv would.  Gates below kLeastGate count as that here,
// zeros too: it is divided out again, and what else they scale is below FP32's rounding.
//
// Three products of 64 tokens with a state and four of the tokens with one another, as warp-wide TF32 products of numbers in two parts (one, for
// BF16 inputs): a warp has 16 rows and 32 columns of a tile of 64 x 64, and the next 16 rows of each operand are in flight meanwhile.
// Bound by shared memory and the splits' instructions: FP32 B4 H16 T1024, 128 x 128, 279 us of the gradients' 1597 (with FP32 multiply-adds, 4 x 4
// numbers per thread, 370).  The sweeps that leave the states write 2 r dv FP32 words per chunk and head, 15 us each there.
constexpr int kGateThreads = 256;

// c += A B for 8 columns and a step of 8.  A1, B1: BF16 numbers, which have no low part.  The tensor cores cut their sums off instead of rounding
// them, so that a long sum would shrink: every step starts at 0 and is added in FP32.
template <bool A1, bool B1>
__device__ __forceinline__ void gate_product(float (&c)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4], const uint32_t (&bh)[2], const uint32_t (&bl)[2])
{
    float d[4] = {};
    if (!A1) mma_tf32(d, al, bh[0], bh[1]);
    if (!B1) mma_tf32(d, ah, bl[0], bl[1]);
    mma_tf32(d, ah, bh[0], bh[1]);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] += d[i];
}

template <bool BF16>
__global__ void __launch_bounds__(kGateThreads, 2)
gdelta_gate_kernel(GdeltaShape s, const void *q, const void *k, const void *dy, float scale, const float *e, const float *lam,
                   const float *S, const float *G, float *dalpha)
{
    constexpr int C = kGateC, KS = 16, LDR = KS + 4, LDC = C + 8, NL = C * KS / kGateThreads;   // (strides without bank conflicts)
    __shared__ float ra[C][LDR], rb[C][LDR], rc[C][LDR];      // [token][column]
    __shared__ float ca[KS][LDC], cb[KS][LDC];                // [state row][value column]
    __shared__ float F[C][C + 1], al[C], be[C], as[2][C], bs[2][C], part[kGateThreads / 32];
    const int nch = (s.T + C - 1) / C, c = blockIdx.x % nch, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t4 = lane & 3, row0 = 16 * (warp & 3), half = warp >> 2, col0 = 32 * half;
    const size_t bh = blockIdx.x / nch;
    const size_t key = (bh / s.H * s.Hk + bh % s.H / (s.H / s.Hk)) * s.T + (size_t)c * C, val = bh * s.T + (size_t)c * C;
    const int nt = min(C, s.T - c * C), r = s.r, dv = s.dv;
    const float *Sc = S + (bh * nch + c) * r * dv, *Gc = G + (bh * nch + c) * r * dv;
    if (tid < C) {
        al[tid] = tid < nt ? fmaxf(s.alpha[val + tid], kLeastGate) : 1.f;
        be[tid] = tid < nt && s.beta ? s.beta[val + tid] : 1.f;
    }
    // a thread's share of 16 columns, from u0 on, of the chunk's rows of an array of d columns
    const int ru = tid & 15, rt = tid >> 4, cu = tid >> 6, cd = tid & 63;
    auto rows_at = [&](float (&x)[NL], auto elem, size_t first, int d, int u0) {
#pragma unroll
        for (int m = 0; m < NL; ++m) {
            const int t = rt + 16 * m;
            x[m] = t < nt && u0 + ru < d ? elem((first + t) * d + u0 + ru) : 0.f;
        }
    };
    auto put_rows = [&](float (*to)[LDR], const float (&x)[NL]) {
#pragma unroll
        for (int m = 0; m < NL; ++m) to[rt + 16 * m][ru] = x[m];
    };
    auto q_at = [&](size_t i) { return load_elem<BF16>(q, i); };
    auto k_at = [&](size_t i) { return load_elem<BF16>(k, i); };
    auto dy_at = [&](size_t i) { return load_elem<BF16>(dy, i); };
    auto e_at = [&](size_t i) { return e[i]; };
    auto lam_at = [&](size_t i) { return lam[i]; };
    // operands of a step of 8: this warp's rows, 8 columns from tokens' rows, 8 columns of a state
    auto left = [&](const float (*from)[LDR], int k0, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) split_tf32_near(from[row0 + g + 8 * (i & 1)][k0 + t4 + 4 * (i >> 1)], hi[i], lo[i]);
    };
    auto right_rows = [&](const float (*from)[LDR], int k0, int n, uint32_t (&hi)[2], uint32_t (&lo)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) split_tf32_near(from[col0 + 8 * n + g][k0 + t4 + 4 * i], hi[i], lo[i]);
    };
    auto right_state = [&](const float (*from)[LDC], int k0, int n, uint32_t (&hi)[2], uint32_t (&lo)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) split_tf32_near(from[k0 + t4 + 4 * i][col0 + 8 * n + g], hi[i], lo[i]);
    };
    __syncthreads();

    // the tokens with the state before the chunk and the gradient behind it
    float av[2] = {}, bv[2] = {}, anchor = 0.f;
    float n0[NL], n1[NL], n2[NL], n3[NL];
    const int usteps = (r + KS - 1) / KS, steps = usteps * ((dv + C - 1) / C);
    auto fetch_states = [&](int i) {
        const int u0 = i % usteps * KS, d = i / usteps * C + cd;
        rows_at(n0, q_at, key, r, u0);
        rows_at(n1, k_at, key, r, u0);
#pragma unroll
        for (int m = 0; m < NL; ++m) {
            const int u = u0 + cu + 4 * m;
            const bool in = u < r && d < dv;
            const size_t at = (size_t)u * dv + d;
            n2[m] = in ? Sc[at] : 0.f, n3[m] = in ? Gc[at] : 0.f;
        }
    };
    fetch_states(0);
    for (int i0 = 0; i0 < steps; i0 += usteps) {
        float qs[4][4] = {}, ks[4][4] = {}, kg[4][4] = {};
        for (int i = i0; i < i0 + usteps; ++i) {
            put_rows(ra, n0);
            put_rows(rb, n1);
#pragma unroll
            for (int m = 0; m < NL; ++m) {
                ca[cu + 4 * m][cd] = n2[m], cb[cu + 4 * m][cd] = n3[m];
                anchor = fmaf(n2[m], n3[m], anchor);
            }
            __syncthreads();
            if (i + 1 < steps) fetch_states(i + 1);
#pragma unroll
            for (int k0 = 0; k0 < KS; k0 += 8) {
                uint32_t qh[4], ql[4], kh[4], kl[4];
                left(ra, k0, qh, ql);
                left(rb, k0, kh, kl);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    uint32_t sh[2], sl[2], gh[2], gl[2];
                    right_state(ca, k0, n, sh, sl);
                    right_state(cb, k0, n, gh, gl);
                    gate_product<BF16, false>(qs[n], qh, ql, sh, sl);
                    gate_product<BF16, false>(ks[n], kh, kl, sh, sl);
                    gate_product<BF16, false>(kg[n], kh, kl, gh, gl);
                }
            }
            __syncthreads();
        }
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = row0 + g + 8 * (j >> 1), d = i0 / usteps * C + col0 + 8 * n + 2 * t4 + (j & 1);
                const bool in = t < nt && d < dv;
                const size_t at = (val + t) * dv + d;
                const float y = in ? dy_at(at) : 0.f, l = in ? lam[at] : 0.f, er = in ? e[at] : 0.f;
                av[j >> 1] = fmaf(scale * qs[n][j], y, fmaf(-be[t] * ks[n][j], l, av[j >> 1]));
                bv[j >> 1] = fmaf(be[t] * kg[n][j], er, bv[j >> 1]);
            }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 2; o; o >>= 1) {
            av[i] += __shfl_xor_sync(0xffffffffu, av[i], o);
            bv[i] += __shfl_xor_sync(0xffffffffu, bv[i], o);
        }
        if (t4 == 0) as[half][row0 + g + 8 * i] = av[i], bs[half][row0 + g + 8 * i] = bv[i];
    }
    anchor = warp_sum(anchor);
    if (lane == 0) part[warp] = anchor;

    // the tokens with one another, where a column of the warp's is not behind all its rows
    const int blocks = min(4, max(0, (row0 + 16 - col0) / 8));
    float qk[4][4] = {}, kk[4][4] = {}, ye[4][4] = {}, le[4][4] = {};
    rows_at(n0, q_at, key, r, 0);
    rows_at(n1, k_at, key, r, 0);
    for (int u0 = 0; u0 < r; u0 += KS) {
        put_rows(ra, n0);
        put_rows(rb, n1);
        __syncthreads();
        if (u0 + KS < r) {
            rows_at(n0, q_at, key, r, u0 + KS);
            rows_at(n1, k_at, key, r, u0 + KS);
        }
        if (blocks)
#pragma unroll
            for (int k0 = 0; k0 < KS; k0 += 8) {
                uint32_t qh[4], ql[4], kh[4], kl[4];
                left(ra, k0, qh, ql);
                left(rb, k0, kh, kl);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    if (n >= blocks) break;
                    uint32_t jh[2], jl[2];
                    right_rows(rb, k0, n, jh, jl);
                    gate_product<BF16, BF16>(qk[n], qh, ql, jh, jl);
                    gate_product<BF16, BF16>(kk[n], kh, kl, jh, jl);
                }
            }
        __syncthreads();
    }
    rows_at(n0, dy_at, val, dv, 0);
    rows_at(n1, lam_at, val, dv, 0);
    rows_at(n2, e_at, val, dv, 0);
    for (int u0 = 0; u0 < dv; u0 += KS) {
        put_rows(ra, n0);
        put_rows(rb, n1);
        put_rows(rc, n2);
        __syncthreads();
        if (u0 + KS < dv) {
            rows_at(n0, dy_at, val, dv, u0 + KS);
            rows_at(n1, lam_at, val, dv, u0 + KS);
            rows_at(n2, e_at, val, dv, u0 + KS);
        }
        if (blocks)
#pragma unroll
            for (int k0 = 0; k0 < KS; k0 += 8) {
                uint32_t yh[4], yl[4], lh[4], ll[4];
                left(ra, k0, yh, yl);
                left(rb, k0, lh, ll);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    if (n >= blocks) break;
                    uint32_t eh[2], el[2];
                    right_rows(rc, k0, n, eh, el);
                    gate_product<BF16, false>(ye[n], yh, yl, eh, el);
                    gate_product<false, false>(le[n], lh, ll, eh, el);
                }
            }
        __syncthreads();
    }
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = row0 + g + 8 * (j >> 1), u = col0 + 8 * n + 2 * t4 + (j & 1);
            F[t][u] = be[u] * fmaf(scale * qk[n][j], ye[n][j], -be[t] * kk[n][j] * le[n][j]);
        }
    __syncthreads();
    // F, and in its place its sums over j < t; the row of the gradient behind the chunk in bs
    if (tid < C) {
        float m = al[tid];
#pragma unroll 4
        for (int j = tid - 1; j >= 0; --j) {
            F[tid][j] *= m;
            m *= al[j];
        }
        float sum = (as[0][tid] + as[1][tid]) * m;
#pragma unroll 4
        for (int t = 0; t <= tid; ++t) {
            const float f = F[tid][t];
            F[tid][t] = sum;
            sum += f;
        }
    } else if (tid == C) {
        float m = 1.f, sum = 0.f;
#pragma unroll 4
        for (int j = C - 1; j >= 0; --j) {
            bs[0][j] = (bs[0][j] + bs[1][j]) * m;
            m *= al[j];
        }
        for (int w = 0; w < kGateThreads / 32; ++w) sum += part[w];
        sum *= m;
#pragma unroll 4
        for (int t = 0; t < C; ++t) {
            const float f = bs[0][t];
            bs[0][t] = sum;
            sum += f;
        }
    }
    __syncthreads();
    if (tid < nt) {
        float sum = bs[0][tid];
#pragma unroll 4
        for (int t = tid; t < C; ++t) sum += F[t][tid];
        dalpha[val + tid] = s.alpha[val + tid] > 0.f ? sum / al[tid] : 0.f;
    }
}

// ------------------------------------------------------------ decode step
// With p = S^T k of the state as it is: e = v - alpha p, S <- alpha S + k (beta e)^T, y = scale S^T q of the rows as they are
// written.  Reads and rewrites r dv FP32 words per head, four FMAs each: bound by HBM.  CTA (b, h, 128 columns) of 8
// warps; a warp takes RW rows, its lanes 4 columns each, issues every state load before any arithmetic and keeps the rows in
// registers.  No store can leave before all of a head's rows are there, so it is other CTAs that keep HBM busy
// meanwhile: at 80 registers three fit an SM (537 MB of state, B = 256 H = 16 128 x 128: 87 us, 6.1 TB/s; two at 128
// registers 96; a ring of three whole states in shared memory, filled and emptied by bulk copies, 98).  So k, q, v and the gates are read
// from shared memory where they are used, and the read of S^T q waits for the write instead of taking registers beside p.
__device__ __forceinline__ float4 ld_stream(const float4 *p)
{
    float4 v;
    asm volatile("ld.global.L1::no_allocate.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ void st_stream(float4 *p, float4 v)
{
    asm volatile("st.global.cs.v4.f32 [%0], {%1,%2,%3,%4};" ::"l"(p), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

__device__ __forceinline__ float4 fma4(float a, float4 x, float4 y)
{
    return make_float4(fmaf(a, x.x, y.x), fmaf(a, x.y, y.y), fmaf(a, x.z, y.z), fmaf(a, x.w, y.w));
}

__device__ __forceinline__ float2 lds_pair(uint32_t a)      // (volatile: not kept in registers from one use to the next)
{
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
    return v;
}

template <bool BF16, int RW>
__global__ void __launch_bounds__(256, RW == 8 ? 5 : RW == 16 ? 3 : 1)
gdelta_decode_kernel(const void *__restrict__ q, const void *__restrict__ k, const void *__restrict__ v, GdeltaShape s,
                     float *__restrict__ S, float scale, void *__restrict__ y)
{
    __shared__ float2 kqs[8 * RW];           // k, q
    __shared__ float4 vs[32];
    __shared__ float2 gates;
    __shared__ float4 part[8][32], part_y[8][32];
    const int r = s.r, dv = s.dv;
    const size_t bh = blockIdx.x, kh = bh / s.H * s.Hk + (bh % s.H) / (s.H / s.Hk);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int j = blockIdx.y * 128 + 4 * lane;
    const bool col = j < dv;
    float4 *Sr = reinterpret_cast<float4 *>(S + (bh * r + (size_t)warp * RW) * dv + (col ? j : 0));
    const int dv4 = dv >> 2;
    float4 x[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (col && warp * RW + i < r) x[i] = ld_stream(Sr + (size_t)i * dv4);
    }
    for (int i = tid; i < 8 * RW; i += 256)
        kqs[i] = i < r ? make_float2(load_elem<BF16>(k, kh * r + i), load_elem<BF16>(q, kh * r + i)) : make_float2(0.f, 0.f);
    if (tid < 128) {
        const int c = blockIdx.y * 128 + tid;
        reinterpret_cast<float *>(vs)[tid] = c < dv ? load_elem<BF16>(v, bh * dv + c) : 0.f;
    }
    if (tid == 0) gates = make_float2(s.alpha ? s.alpha[bh] : 1.f, s.beta ? s.beta[bh] : 1.f);
    __syncthreads();
    const uint32_t kq0 = smem_u32(kqs + warp * RW);
    float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < RW; ++i) c = fma4(lds_pair(kq0 + 8 * i).x, x[i], c);
    part[warp][lane] = c;
    __syncthreads();
    c = part[0][lane];
#pragma unroll
    for (int w = 1; w < 8; ++w) c = fma4(1.f, part[w][lane], c);
    const float al = gates.x;
    {
        const float be = gates.y;
        const float4 vv = vs[lane];
        c = make_float4(be * fmaf(-al, c.x, vv.x), be * fmaf(-al, c.y, vv.y), be * fmaf(-al, c.z, vv.z), be * fmaf(-al, c.w, vv.w));
    }
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        const float2 kq = lds_pair(kq0 + 8 * i);
        const float4 n = make_float4(fmaf(al, x[i].x, kq.x * c.x), fmaf(al, x[i].y, kq.x * c.y), fmaf(al, x[i].z, kq.x * c.z),
                                     fmaf(al, x[i].w, kq.x * c.w));
        if (col && warp * RW + i < r) st_stream(Sr + (size_t)i * dv4, n);
        u = fma4(kq.y, n, u);
    }
    part_y[warp][lane] = u;
    __syncthreads();
    if (warp == 0 && col) {
#pragma unroll
        for (int w = 1; w < 8; ++w) u = fma4(1.f, part_y[w][lane], u);
        store_elem<BF16>(y, bh * dv + j, scale * u.x);
        store_elem<BF16>(y, bh * dv + j + 1, scale * u.y);
        store_elem<BF16>(y, bh * dv + j + 2, scale * u.z);
        store_elem<BF16>(y, bh * dv + j + 3, scale * u.w);
    }
}

template <bool BF16>
cudaError_t launch_dec(const GdeltaShape &s, const void *q, const void *k, const void *v, float *S, float scale, void *y,
                       cudaStream_t stream)
{
    const dim3 grid((unsigned)(s.B * s.H), (s.dv + 127) / 128);
    if (s.r <= 64) gdelta_decode_kernel<BF16, 8><<<grid, 256, 0, stream>>>(q, k, v, s, S, scale, y);
    else if (s.r <= 128) gdelta_decode_kernel<BF16, 16><<<grid, 256, 0, stream>>>(q, k, v, s, S, scale, y);
    else gdelta_decode_kernel<BF16, 32><<<grid, 256, 0, stream>>>(q, k, v, s, S, scale, y);
    return cudaGetLastError();
}

}  // namespace

// Segments of a dense forward call (1: none) on `sms` SMs: the least of the estimates, in us, of one pass over the tokens and of two
// passes over a segment's (5 of set-up each, 8 between the launches) with a join per segment (1.6 + r / 40 up to 64 rows, else 1.6 + r / 64 for each 32), as long as
// the first pass's CTAs, N's and M's columns, find an SM each.  Whole and in segments: B2 H4 T1001, 64 x 96 104 and 84 us, T4096 406 and 284;
// one head of 8192 tokens, 128 x 128, 1285 and 391.  Segments are whole blocks of tokens.
int gdelta_rec_segments(int B, int H, int T, int r, int dv, int sms)
{
    const long long ctas = (long long)B * H * ((dv + kRecCols - 1) / kRecCols + (r + kRecCols - 1) / kRecCols);
    const double token = r <= 64 ? 0.101 : r <= 128 ? 0.157 : 0.23, join = r <= 64 ? 1.6 + r / 40.0 : (1.6 + r / 64.0) * ((r + 31) / 32);
    if (T == 0) return 1;
    int best = 1;
    double least = T * token;
    for (int n = 2; n <= 16 && n * ctas <= sms + sms / 8; ++n) {
        const int len = ((T + n - 1) / n + kRecTok - 1) / kRecTok * kRecTok, used = (T + len - 1) / len;
        const double t = 2 * (len * token + 5) + 8 + (used - 1) * join;
        if (used == n && t < least) least = t, best = n;
    }
    return best;
}

size_t gdelta_rec_floats(int B, int H, int T, int r, int dv, int sms)
{
    const int n = gdelta_rec_segments(B, H, T, r, dv, sms);
    return n > 1 ? (size_t)B * H * n * r * (2 * (size_t)dv + r) : 0;
}

cudaError_t launch_gdelta_rec_segments(const GdeltaShape &s, const GdeltaForward &f, bool bf16, int sms, float *ws, cudaStream_t stream)
{
    const int n = gdelta_rec_segments(s.B, s.H, s.T, s.r, s.dv, sms);
    if (n == 1) return launch_gdelta_rec(s, f, bf16, stream);
    static OncePerDevice once;
    const uint32_t rp = (s.r + 3) & ~3;
    cudaError_t e = set_smem_once(gdelta_join_kernel<4, 8>, 3 * 256 * 32 * 4, once);
    if (e != cudaSuccess) return e;
    RecArgs a{};
    a.s = s;
    a.q = f.q, a.k = f.k, a.v = f.v;
    a.scale = f.scale;
    a.nseg = n, a.seg_len = ((s.T + n - 1) / n + kRecTok - 1) / kRecTok * kRecTok;
    const size_t state = (size_t)s.B * s.H * n * s.r * s.dv;
    a.N = ws, a.M = ws + 2 * state, a.starts = ws + state;
    a.sums = true;
    if ((e = launch_rec<kFwd>(a, bf16, stream)) != cudaSuccess) return e;
    // up to 64 rows in one step (B2 H4 T1001, 64 x 96: 90 us by 32 at a time, 84 so)
    const bool one = s.r <= 64;
    e = launch_after(one ? gdelta_join_kernel<8, 2> : gdelta_join_kernel<4, 8>, dim3((s.dv + 31) / 32, s.B * s.H), 256,
                     (one ? 128 : 96) * rp * 4, stream, s, f.S0, a.N, a.M, ws + state, n);
    if (e != cudaSuccess) return e;
    a.sums = false;
    a.y = f.y, a.S_fin = f.S_out;
    return launch_rec<kFwd>(a, bf16, stream);
}

cudaError_t launch_gdelta_rec(const GdeltaShape &s, const GdeltaForward &f, bool bf16, cudaStream_t stream)
{
    RecArgs a{};
    a.s = s;
    a.q = f.q, a.k = f.k, a.v = f.v, a.y = f.y;
    a.S_init = f.S0, a.S_fin = f.S_out;
    a.scale = f.scale;
    return launch_rec<kFwd>(a, bf16, stream);
}

cudaError_t launch_gdelta_decode(const GdeltaShape &s, const void *q, const void *k, const void *v, bool bf16, float *S,
                                 float scale, void *y, cudaStream_t stream)
{
    return bf16 ? launch_dec<true>(s, q, k, v, S, scale, y, stream) : launch_dec<false>(s, q, k, v, S, scale, y, stream);
}

cudaError_t launch_gdelta_group_sum(const GdeltaShape &s, const float *dq, const float *dk, bool bf16, void *dq_out, void *dk_out,
                                    cudaStream_t stream)
{
    const unsigned grid = (unsigned)(((long long)s.B * s.Hk * s.T * s.r + 255) / 256);
    return launch_after(bf16 ? gdelta_group_sum_kernel<true> : gdelta_group_sum_kernel<false>, grid, 256, 0, stream, s, dq, dk, dq_out,
                        dk_out);
}

// e, lam [B,H,T,dv]; w (then dk), dq [B,H,T,r]; the states before every chunk and the gradients behind it
size_t gdelta_rec_backward_floats(int B, int H, int T, int r, int dv)
{
    const size_t heads = (size_t)B * H, chunks = (T + (size_t)kGateC - 1) / kGateC;
    return heads * T * (2 * (size_t)dv + 2 * (size_t)r) + heads * chunks * 2 * r * dv;
}

cudaError_t launch_gdelta_rec_backward(const GdeltaShape &s, const GdeltaBackward &g, bool bf16, cudaStream_t stream)
{
    const size_t heads = (size_t)s.B * s.H, tokens = heads * s.T, chunks = heads * ((s.T + kGateC - 1) / kGateC);
    float *e = g.ws, *lam = e + tokens * s.dv, *w = lam + tokens * s.dv, *dq = w + tokens * s.r, *S = dq + tokens * s.r,
          *G = S + chunks * s.r * s.dv;
    const bool gates = s.alpha && g.dalpha;
    RecArgs a{};
    a.s = s;
    a.q = g.q, a.k = g.k, a.v = g.v, a.dy = g.dy;
    a.scale = g.scale;
    a.e = a.e_out = e, a.lam = a.lam_out = lam;
    a.w = w, a.dq = dq, a.dv_out = g.dv_out;
    cudaError_t st = cudaSuccess;
    a.S_init = g.S0, a.ckpt = gates ? S : nullptr;
    if ((st = launch_rec<kFwd>(a, bf16, stream)) != cudaSuccess) return st;
    a.S_init = g.dS_T, a.S_fin = g.dS0, a.ckpt = gates ? G : nullptr;
    if ((st = launch_rec<kRev>(a, bf16, stream)) != cudaSuccess) return st;
    a.S_fin = a.ckpt = nullptr;
    a.S_init = g.S0;
    if ((st = launch_rec<kQue>(a, bf16, stream)) != cudaSuccess) return st;
    a.S_init = g.dS_T;
    if ((st = launch_rec<kKey>(a, bf16, stream)) != cudaSuccess) return st;
    if (g.dbeta) gdelta_beta_kernel<<<(unsigned)((tokens + 7) / 8), 256, 0, stream>>>(s, lam, e, g.dbeta);
    if ((st = launch_gdelta_group_sum(s, dq, w, bf16, g.dq, g.dk, stream)) != cudaSuccess) return st;
    if (gates)
        (bf16 ? gdelta_gate_kernel<true> : gdelta_gate_kernel<false>)<<<(unsigned)chunks, kGateThreads, 0, stream>>>(
            s, g.q, g.k, g.dy, g.scale, e, lam, S, G, g.dalpha);
    return cudaGetLastError();
}

}  // namespace la
