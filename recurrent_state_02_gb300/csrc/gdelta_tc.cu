// gdelta_tc.cu -- the gated delta rule chunk by chunk on the tensor cores (BF16 inputs, FP32 state).
//
// With G_i the running sum of log alpha inside a chunk of C = 64 tokens and S the state before it, the errors
// e_i = v_i - S'^T k_i that the rule writes solve, row by row,
//     (I + L) E = R,   R = V - e^G K S,   L_ij = e^{G_i - G_j} (k_i . k_j) beta_j  (j < i),
// so with X = (I + L)^{-1} (unit lower triangular, known from k and the gates alone) and V' = beta E
//     E = X R,   Y = scale (e^G Q S + A V'),   S_next = e^{G_C} S + K^T (e^{G_C - G} V'),   A_ij = e^{G_i - G_j} q_i . k_j  (j <= i).
// Every exponent is a difference that is <= 0.
//
// A first kernel (gdelta_prep_kernel, one CTA per chunk and head) forms A, X and the gates; the second one
// (gdelta_chain_kernel, one CTA per head and 128 value columns) carries the state.  It works on transposes: S^T has a value
// column per TMEM lane, so that the products' left operands (S^T, R^T, V'^T) are what a thread has just computed
// for its lane and go back to TMEM as they are, never through shared memory; K, Q, X and A are right operands in the
// layout in which they arrive.  Per chunk
//     1  P^T = S^T K^T                     R^T = V^T - e^G P^T
//     2  E^T = R^T X^T                     V'^T = beta E^T
//     3  dS^T = (e^{G_C - G} V'^T) K       S^T = e^{G_C} S^T + dS^T
// and off the chain  Q S  after 2 and  A V'  after 3, which the threads turn into y during the next chunk's step 1.
//
// Precision: the state lives in FP32 registers.  q, k, v are exact as BF16 operands; what the kernels derive is split into
// two BF16 parts (16 bits of mantissa and a sign) wherever it reaches the state -- S, R, X and V' in steps 1 to 3, the product of
// two such parts' low halves left out -- and is rounded to one where it reaches y only (which is BF16).  Against 64 bits the
// state is off by 4e-6 and y by 2.7e-3 (relative 2-norms at B4 H16 T4096; the rounding of y alone is 1.7e-3).

#include "gdelta_tc.cuh"
#include "mma_tf32.cuh"

namespace la {
namespace {

// ------------------------------------------------------------------- the plan
// Packed sequences, one CTA: checks the bounds, numbers the chunks (slot_base[b], slot_base[B] = their count)
// and ranks the sequences, longest first (order), so that a long one does not start last.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads)
gdelta_plan_kernel(const int *cu, int B, int total, int *slot_base, int *order, int *status)
{
    __shared__ int part[32], len[kPlanThreads];
    let_next_start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int carry = 0;
    for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int n = 0;
        bool ok = false;
        if (b < B) {
            const int lo = cu[b], hi = cu[b + 1];
            ok = lo >= 0 && hi >= lo && hi <= total;
            if (ok) n = (hi - lo + kC - 1) / kC;
            else atomicExch(status, kStatusShape);
        }
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) part[warp] = x;
        len[tid] = ok ? n : -1;
        __syncthreads();
        int before = carry, all = 0;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) before += part[w];
            all += part[w];
        }
        // (sequences that overlap may add up to more chunks than the workspace holds: the rest is left out)
        if (b < B) slot_base[b] = ok && before + x <= total / kC + B ? before + x - n : -1;
        if (ok && before + x > total / kC + B) atomicExch(status, kStatusShape);
        if (B <= kPlanThreads && b < B) {
            int rank = 0;
            for (int i = 0; i < B; ++i) rank += len[i] > len[tid] || (len[i] == len[tid] && i < tid);
            order[rank] = b;
        } else if (b < B) {
            order[b] = b;
        }
        carry += all;
        __syncthreads();
    }
    if (tid == 0) slot_base[B] = min(carry, total / kC + B);
}

// Up to 32 sequences need no plan kernel (16 short ones as a graph: 27 us with it, 23 without): every warp finds its own, sequence b in lane b.
// Returns the sequence that holds chunk `want` (CHUNK), or the one of rank `want`, longest first; -1 is none.
constexpr int kSelfPlan = 32;
template <bool CHUNK>
__device__ __forceinline__ int self_plan(const GdeltaTcArgs &a, int want, Span &sp)
{
    const int lane = threadIdx.x & 31, B = a.s.B;
    int lo = 0, T = 0, n = -1;
    if (lane < B) {
        lo = a.s.cu_seqlens[lane];
        const int hi = a.s.cu_seqlens[lane + 1];
        if (lo >= 0 && hi >= lo && hi <= a.s.T) T = hi - lo, n = (T + kC - 1) / kC;
    }
    int behind = max(n, 0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, behind, o);
        if (lane >= o) behind += x;
    }
    const int base = behind - max(n, 0);
    const bool valid = n >= 0 && behind <= a.s.T / kC + B;
    if (lane < B && !valid && !CHUNK && blockIdx.x == 0) atomicExch(a.s.status, kStatusShape);
    bool mine;
    if (CHUNK) {
        mine = valid && base <= want && want < behind;
    } else {
        int rank = 0;
        for (int i = 0; i < B; ++i) {
            const int other = __shfl_sync(0xffffffffu, n, i);
            rank += other > n || (other == n && i < lane);
        }
        mine = lane < B && rank == want;
    }
    const uint32_t v = __ballot_sync(0xffffffffu, mine);
    if (!v) return -1;
    const int b = __ffs(v) - 1;
    sp.valid = __shfl_sync(0xffffffffu, (int)valid, b);
    sp.tok0 = __shfl_sync(0xffffffffu, lo, b);
    sp.T = __shfl_sync(0xffffffffu, T, b);
    sp.slot = __shfl_sync(0xffffffffu, base, b);
    return b;
}

// ------------------------------------------------------- A, X and the gates
// Four warps per chunk and head.  [G; P] = [K; Q] K^T on the tensor cores; a row of L or A per thread, its decays as running products
// of the gates from the diagonal to the left (no logarithms, and gates of 0 need no care); then X = (I + L)^{-1} in FP32: the four
// diagonal blocks of 16 by forward substitution, two in a warp, and the blocks below them, 16 and then 32 wide, as
// X_10 = -X_11 (L_10 X_00) in warp-wide TF32 products of numbers in two parts.  (As FP32 sums with 2 x 2 and 4 x 2 numbers per thread
// these products took 60 % of the kernel's 4000 shared-memory wavefronts per chunk, which bound it.)
// Now 2100 instructions per warp and chunk: 55 us for 4096 chunks (B4 H16 T4096, 128 wide; 76 before), issue slots and shared
// memory 55 % busy, the rest being the solve's barriers at 24 warps per SM.  For the gradients 75 us, half of HBM's rate.
constexpr int kPThreads = 128;
// FP32 row strides of Lt, of the 32 x 32 blocks and of the 16 x 16 ones: the operands of the small products are read without
// bank conflicts
constexpr int LD = 72, LDT = 40, LDS16 = 24;
// K and Q interleaved by 64-feature block ([K; Q] is one 128-row operand per block); once [G; P] is complete the region
// holds L and the solve's blocks
constexpr uint32_t kPL = 0;                      // Lt (64 x LD): Lt[u][i] holds row i, column u; then X10 [i][j]
constexpr uint32_t kPX00 = kPL + kC * LD * 4;    // X00 [u][j]
constexpr uint32_t kPX11t = kPX00 + 32 * LDT * 4;   // X11 transposed [u][i]
constexpr uint32_t kPM = kPX11t + 32 * LDT * 4;  // M = L10 X00 [u][j]; before it the same for the two 32-blocks' halves
constexpr uint32_t kPA = kPX00;                  // before them A's image (BACK: two), on its way out
constexpr uint32_t kPGate = kPA + 2 * kTile;     // alpha, beta and e^G of the chunk's tokens
static_assert(2 * 16 * LDS16 <= 32 * LDT, "the halves' products fit");
constexpr uint32_t kPSmall = kPGate + 3 * kC * 4;
static_assert(kPGate >= 4 * kTile && kPGate >= kPM + 32 * LDT * 4 && kPGate % 16 == 0, "the gates lie behind the K, Q tiles and the blocks");

struct alignas(16) PSmall {
    uint64_t full, mma;
    uint32_t tmem_base;
    int abort_flag;
};
constexpr uint32_t kPSmemBytes = kPSmall + sizeof(PSmall) + 1024;

// A warp: c += A B, A 16 x 8 K8 (element (row, k) = a(row, k)), B 8 K8 x 8 N, in FP32 but for the product of the low parts (2^-20
// of the terms; X goes on as two BF16 parts, 2^-17).  c[n][0..3]: rows lane / 4 (+ 8), columns 8 n + 2 (lane % 4) (+ 1) as (row, col), (row, col + 1), (row + 8, ..)
template <int K8, int N, class A, class B>
__device__ __forceinline__ void small_product(float (&c)[N][4], int lane, A a, B b)
{
    const int g = lane >> 2, t = lane & 3;
#pragma unroll 1               // (unrolled, the kernel waits for instructions)
    for (int k = 0; k < 8 * K8; k += 8) {
        uint32_t ah[4], al[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_tf32(a(g + 8 * (i & 1), k + t + 4 * (i >> 1)), ah[i], al[i]);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            uint32_t bh[2], bl[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) split_tf32(b(k + t + 4 * i, 8 * n + g), bh[i], bl[i]);
            mma_tf32(c[n], al, bh[0], bh[1]);
            mma_tf32(c[n], ah, bl[0], bl[1]);
            mma_tf32(c[n], ah, bh[0], bh[1]);
        }
    }
}

// BACK: for the gradients, which take A in two parts and betas of at least 2^-40 (dbeta is formed by dividing by them; the
// change is far below FP32's rounding).
constexpr float kLeastBeta = 9.094947017729282e-13f;
template <int KD, bool BACK>
__global__ void __launch_bounds__(kPThreads, 6)
gdelta_prep_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k, const GdeltaTcArgs args)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = align1024(smem_raw);
    PSmall *sm = reinterpret_cast<PSmall *>(base + kPSmall);
    float *Lt = reinterpret_cast<float *>(base + kPL);
    float *X10 = Lt;
    float *X00 = reinterpret_cast<float *>(base + kPX00);
    float *X11t = reinterpret_cast<float *>(base + kPX11t);
    float *Mf = reinterpret_cast<float *>(base + kPM);
    float *alpha = reinterpret_cast<float *>(base + kPGate), *beta = alpha + kC, *expG = beta + kC;

    const GdeltaShape &s = args.s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool packed = s.cu_seqlens != nullptr;
    const bool planned = args.slot_base != nullptr;
    if (planned) wait_for_last();
    // this CTA's head, sequence and chunk
    const int h = blockIdx.x % s.H, hk = h / (s.H / s.Hk);
    int slot = blockIdx.x / s.H;
    int b, c;
    Span sp;
    if (packed && !planned) {
        b = self_plan<true>(args, slot, sp);
        if (b < 0) return;
        c = slot - (int)sp.slot;
    } else if (packed) {
        if (slot >= args.slot_base[s.B]) return;
        // the last sequence that starts at or before the slot, 32 probes at a time (-1: skipped ones are passed over)
        int lo = 0, n = s.B;
        while (n > 0) {
            const int step = (n + 31) / 32, at = lo + lane * step;
            bool before = false;
            if (lane * step < n) {
                int base_at = -1, i = at;
                const int end = min(at + step, lo + n);
                while (i < end && (base_at = args.slot_base[i]) < 0) ++i;
                before = base_at >= 0 && base_at <= slot;
            }
            const uint32_t v = __ballot_sync(0xffffffffu, before);
            const int last = v ? 31 - __clz(v) : 0;
            lo += last * step;
            n = min(step, n - last * step);
            if (step == 1) break;
        }
        b = lo;
        sp = span_of(args, b);
        c = slot - (int)sp.slot;
        if (!sp.valid || c < 0 || c * kC >= sp.T) return;
    } else {
        const int nch = (s.T + kC - 1) / kC, part = args.chunks ? args.chunks : nch;
        b = slot / part, c = args.first + slot % part;
        slot = b * nch + c;
        sp = span_of(args, b);
    }
    const int t0 = c * kC, nt = min(kC, sp.T - t0);
    Ctx cx{&sm->abort_flag, kWaitLimitNs, s.status};

    if (tid == 0) {
        mbar_init(&sm->full, 1);
        mbar_init(&sm->mma, 1);
        sm->abort_flag = 0;
        fence_mbarrier_init();
        mbar_arrive_expect_tx(&sm->full, KD / 64 * 2 * kTile);
#pragma unroll
        for (int x = 0; x < KD / 64; ++x) {
            uint8_t *dst = base + x * 2 * kTile;
            if (packed) {
                tma_load_3d(dst, &map_k, &sm->full, 64 * x, hk, (int)sp.tok0 + t0);
                tma_load_3d(dst + kTile, &map_q, &sm->full, 64 * x, hk, (int)sp.tok0 + t0);
            } else {
                tma_load_3d(dst, &map_k, &sm->full, 64 * x, t0, b * s.Hk + hk);
                tma_load_3d(dst + kTile, &map_q, &sm->full, 64 * x, t0, b * s.Hk + hk);
            }
        }
    }
    if (warp == 1) {
        tmem_alloc(&sm->tmem_base, 64);
        tmem_relinquish();
    }
    uint8_t *wsc = args.ws + ((size_t)slot * s.H + h) * (BACK ? kWsChunkB : kWsChunk);
    if (warp == 0) {
        // lane l: tokens 2 l, 2 l + 1.  e^G and e^{G_C - G} as products from the left and from the right.
        const int i0 = 2 * lane;
        float al[2], be[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = t0 + i0 + e;
            const size_t at = packed ? (sp.tok0 + t) * s.H + h : ((size_t)b * s.H + h) * s.T + t;
            const bool in = i0 + e < nt;
            al[e] = in && s.alpha ? s.alpha[at] : 1.f;
            be[e] = in ? (s.beta ? s.beta[at] : 1.f) : 0.f;
            if (BACK) {
                float ratio = 1.f;
                if (in && fabsf(be[e]) < kLeastBeta) {
                    const float least = copysignf(kLeastBeta, be[e]);
                    ratio = be[e] / least, be[e] = least;
                }
                reinterpret_cast<float *>(wsc + kWsGates + kGateRatio)[i0 + e] = ratio;
            }
        }
        float left = al[0] * al[1], right = left;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, left, o), y = __shfl_down_sync(0xffffffffu, right, o);
            if (lane >= o) left *= x;
            if (lane + o < 32) right *= y;
        }
        float before = __shfl_up_sync(0xffffffffu, left, 1), behind = __shfl_down_sync(0xffffffffu, right, 1);
        if (lane == 0) before = 1.f;
        if (lane == 31) behind = 1.f;
        float2 *g = reinterpret_cast<float2 *>(wsc + kWsGates);
        g[lane] = make_float2(before * al[0], before * al[0] * al[1]);
        g[kC / 2 + lane] = make_float2(al[1] * behind, behind);
        g[kC + lane] = make_float2(be[0], be[1]);
        reinterpret_cast<float2 *>(alpha)[lane] = make_float2(al[0], al[1]);
        reinterpret_cast<float2 *>(beta)[lane] = make_float2(be[0], be[1]);
        if (BACK) {
            reinterpret_cast<float2 *>(expG)[lane] = make_float2(before * al[0], before * al[0] * al[1]);
            // G itself in 64 bits, kept as two FP32 parts: differences over a few tokens stay exact to FP32 behind gates near 0.
            // Gates below kLeastGate count as that there, and how many there are is kept beside: what they scale is 0.
            const double l0 = log2f(fmaxf(al[0], kLeastGate)), l1 = log2f(fmaxf(al[1], kLeastGate));
            double inc = l0 + l1;
            const uint32_t c0 = __ballot_sync(0xffffffffu, al[0] < kLeastGate), c1 = __ballot_sync(0xffffffffu, al[1] < kLeastGate);
            const uint32_t up = 0xffffffffu >> (31 - lane);
            reinterpret_cast<float2 *>(wsc + kWsGates + kGateClosed)[lane] = make_float2(__popc(c0 & up) + __popc(c1 & (up >> 1)),
                                                                                        __popc(c0 & up) + __popc(c1 & up));
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            const double G0 = inc - l1;
            const float h0 = (float)G0, h1 = (float)inc;
            reinterpret_cast<float4 *>(wsc + kWsGates + kGateLog)[lane] = make_float4(h0, (float)(G0 - h0), h1, (float)(inc - h1));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // (the chain's CTAs take all TMEM of an SM and then wait for this kernel: none is placed before every CTA here has its columns)
    let_next_start();
    const uint32_t tmem = sm->tmem_base;

    // [G; P] = [K; Q] K^T (M = 128: G in TMEM lanes 0..63, P in lanes 64..127)
    bool ok = true, issued = false;
    if (warp == 1) {
        ok = warp_wait(cx, &sm->full, 0);
        if (ok && elect_one()) {
            tc_fence_after();
            constexpr uint32_t id = idesc_bf16_f32(128, 64, false, false);
            const uint32_t klo = desc_lo(smem_u32(base), 16);
#pragma unroll
            for (int kk = 0; kk < KD / 16; ++kk) {
                const uint32_t o = ((kk >> 2) * 2 * kTile + (kk & 3) * 32) >> 4;
                mma_ss(tmem, klo + o, kHi128, klo + o, kHi128, id, kk > 0);
            }
            tc_commit(&sm->mma);
        }
        issued = ok;
        __syncwarp();
    }
    if (BACK) {
        // scale e^G Q, 16-byte words of its tiles
        ok = warp_wait(cx, &sm->full, 0) && ok;
        if (ok) {
#pragma unroll 2
            for (int x = tid; x < KD / 64 * 8 * kC; x += kPThreads) {
                const int row = (x >> 3) & 63;
                const uint32_t o = sw128_offset(row, x & 7);
                const uint4 q4 = *reinterpret_cast<const uint4 *>(base + (x >> 9) * 2 * kTile + kTile + o);
                const float f = args.scale * expG[row];
                const uint32_t qw[4] = {q4.x, q4.y, q4.z, q4.w};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) split(__fmul2_rn(make_float2(f, f), make_float2(bf16_lo(qw[e]), bf16_hi(qw[e]))), hi[e], lo[e]);
                uint8_t *to = wsc + kWsQ + (x >> 9) * kTile + o;
                *reinterpret_cast<uint4 *>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(to + KD / 64 * kTile) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        }
    }
    ok = warp_wait(cx, &sm->mma, 0) && ok;
    tc_fence_after();
    if (!__syncthreads_or(!ok)) {
        // Warps 0, 1 (TMEM lanes 0..63): row ri of L, transposed into Lt.  Warps 2, 3: row ri of A, as its image.  Rows past the
        // sequence's end (which hold another one's tokens) count as 0.
        {
            const int ri = 32 * (warp & 1) + lane;
            const uint32_t tq = tmem + ((uint32_t)(32 * warp) << 16);
            const bool real = ri < nt;
            uint8_t *arow = base + kPA + ri * 128, *lrow = arow + kTile;
            float dec = 1.f, next = 1.f;         // e^{G_i - G_j}; the gate of token j + 1
#pragma unroll 1
            for (int half = warp & 1; half >= 0; --half) {
                float v[32];
                tc_ld_32x32b_x32(tq + 32 * half, v);
                wait_loaded(v);
#pragma unroll
                for (int x = 3; x >= 0; --x) {
#pragma unroll
                    for (int y = 1; y >= 0; --y) {
                        const int j0 = 32 * half + 8 * x + 4 * y;
                        const float4 a4 = *reinterpret_cast<const float4 *>(alpha + j0),
                                     b4 = warp < 2 ? *reinterpret_cast<const float4 *>(beta + j0) : a4;
                        const float av[4] = {a4.x, a4.y, a4.z, a4.w}, bv[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                        for (int e = 3; e >= 0; --e) {
                            const int j = j0 + e;
                            float &w = v[8 * x + 4 * y + e];
                            dec = j < ri ? dec * next : 1.f;
                            next = av[e];
                            if (warp < 2) Lt[j * LD + ri] = real && j < ri ? dec * bv[e] * w : 0.f;
                            else w = real && j <= ri ? dec * w : 0.f;
                        }
                    }
                    if (warp >= 2) {
                        const uint4 hi = pack8(v + 8 * x);
                        const int word = ((4 * half + x) ^ (ri & 7)) << 4;
                        *reinterpret_cast<uint4 *>(arow + word) = hi;
                        if (BACK) {
                            const uint32_t hw[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) v[8 * x + 2 * e] -= bf16_lo(hw[e]), v[8 * x + 2 * e + 1] -= bf16_hi(hw[e]);
                            *reinterpret_cast<uint4 *>(lrow + word) = pack8(v + 8 * x);
                        }
                    }
                }
            }
            if (warp == 2) {                     // the zeros of A's upper right quarter
#pragma unroll
                for (int x = 4; x < 8; ++x) {
                    *reinterpret_cast<uint4 *>(arow + ((x ^ (ri & 7)) << 4)) = make_uint4(0, 0, 0, 0);
                    if (BACK) *reinterpret_cast<uint4 *>(lrow + ((x ^ (ri & 7)) << 4)) = make_uint4(0, 0, 0, 0);
                }
            }
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 3 * 32) {            // A goes out as it lies (row by row it would take a line per lane)
            bulk_store(wsc + kWsA, smem_u32(base + kPA), kTile);
            if (BACK) bulk_store(wsc + kWsAl, smem_u32(base + kPA) + kTile, kTile);
            asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
        }
        // The diagonal blocks of 16, two in each of the first two warps: lane l + 16 m owns column l of block 2 warp + m; after step
        // u, acc[u] is final and is subtracted from the rows below.
        const int l = lane & 15, o = lane & 16;
        float acc[16];
        if (warp < 2) {
            const float *Lb = Lt + (32 * warp + o) * LD + 32 * warp + o;
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i] = i == l ? 1.f : 0.f;
#pragma unroll
            for (int u = 0; u < 15; ++u) {
                const float t = acc[u];
#pragma unroll
                for (int g4 = (u + 1) >> 2; g4 < 4; ++g4) {
                    const float4 q = *reinterpret_cast<const float4 *>(Lb + u * LD + 4 * g4);
                    const float lv[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (4 * g4 + e > u) acc[4 * g4 + e] = fmaf(-lv[e], t, acc[4 * g4 + e]);
                }
            }
        }
        __syncthreads();                // (A has been read)
        // X00 by rows, X11 by columns, and the zeros above the diagonal
        if (warp == 0) {
#pragma unroll
            for (int u = 0; u < 16; ++u) X00[(o + u) * LDT + o + l] = acc[u];
        } else if (warp == 1) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
                *reinterpret_cast<float4 *>(X11t + (o + l) * LDT + o + 4 * m) = make_float4(acc[4 * m], acc[4 * m + 1], acc[4 * m + 2], acc[4 * m + 3]);
        } else if (warp == 2) {
#pragma unroll
            for (int u = 0; u < 8; ++u) X00[(2 * u + (o >> 4)) * LDT + 16 + l] = 0.f;
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u) X11t[(16 + 2 * u + (o >> 4)) * LDT + l] = 0.f;
        }
        __syncthreads();
        // The blocks of 16 below them, X_b0 = -X_b (L_b0 X_a): two warps per 32-block, 8 columns each.  C's rows and columns of a lane:
        const int r = lane >> 2, c = 2 * (lane & 3);
        {
            const int k2 = warp >> 1, n0 = 8 * (warp & 1);
            float *M = Mf + k2 * 16 * LDS16;
            const float *Lo = Lt + 32 * k2 * LD + 32 * k2 + 16;
            float m[1][4] = {};
            auto lo = [&](int row, int u) { return Lo[u * LD + row]; };
            if (k2 == 0) small_product<2>(m, lane, lo, [&](int u, int col) { return X00[u * LDT + n0 + col]; });
            else small_product<2>(m, lane, lo, [&](int u, int col) { return X11t[(n0 + col) * LDT + u]; });
            *reinterpret_cast<float2 *>(M + r * LDS16 + n0 + c) = make_float2(m[0][0], m[0][1]);
            *reinterpret_cast<float2 *>(M + (r + 8) * LDS16 + n0 + c) = make_float2(m[0][2], m[0][3]);
            __syncthreads();
            float x[1][4] = {};
            auto mb = [&](int u, int col) { return M[u * LDS16 + n0 + col]; };
            if (k2 == 0) {
                small_product<2>(x, lane, [&](int row, int u) { return -X00[(16 + row) * LDT + 16 + u]; }, mb);
                *reinterpret_cast<float2 *>(X00 + (16 + r) * LDT + n0 + c) = make_float2(x[0][0], x[0][1]);
                *reinterpret_cast<float2 *>(X00 + (24 + r) * LDT + n0 + c) = make_float2(x[0][2], x[0][3]);
            } else {
                small_product<2>(x, lane, [&](int row, int u) { return -X11t[(16 + u) * LDT + 16 + row]; }, mb);
#pragma unroll
                for (int e = 0; e < 4; ++e) X11t[(n0 + c + (e & 1)) * LDT + 16 + r + 8 * (e >> 1)] = x[0][e];
            }
        }
        __syncthreads();
        // M = L10 X00 and then X10 = -X11 M: a 16 x 16 quarter per warp
        const int r0 = 16 * (warp >> 1), n0 = 16 * (warp & 1);
        auto put = [&](float *to, const float (&o)[2][4]) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                *reinterpret_cast<float2 *>(to + (r0 + r) * LDT + n0 + 8 * n + c) = make_float2(o[n][0], o[n][1]);
                *reinterpret_cast<float2 *>(to + (r0 + r + 8) * LDT + n0 + 8 * n + c) = make_float2(o[n][2], o[n][3]);
            }
        };
        {
            float m[2][4] = {};
            small_product<4>(m, lane, [&](int row, int u) { return Lt[u * LD + 32 + r0 + row]; },
                             [&](int u, int col) { return X00[u * LDT + n0 + col]; });
            put(Mf, m);
        }
        __syncthreads();
        {
            float x[2][4] = {};
            small_product<4>(x, lane, [&](int row, int u) { return -X11t[u * LDT + r0 + row]; },
                             [&](int u, int col) { return Mf[u * LDT + n0 + col]; });
            put(X10, x);
        }
        __syncthreads();
        // X's two parts, 16-byte words of the images' rows
        uint8_t *xi = wsc + kWsX;
#pragma unroll 1
        for (int x = tid; x < 8 * kC; x += kPThreads) {
            const int row = x >> 3, w = x & 7, r = row & 31, c8 = 8 * (w & 3);
            float v[8] = {};
            if (w < 4) {
                const float *from = (row < 32 ? X00 : X10) + r * LDT + c8;
                const float4 u0 = *reinterpret_cast<const float4 *>(from), u1 = *reinterpret_cast<const float4 *>(from + 4);
                v[0] = u0.x, v[1] = u0.y, v[2] = u0.z, v[3] = u0.w, v[4] = u1.x, v[5] = u1.y, v[6] = u1.z, v[7] = u1.w;
            } else if (row >= 32) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = X11t[(c8 + e) * LDT + r];
            }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split(make_float2(v[2 * e], v[2 * e + 1]), hi[e], lo[e]);
            const uint32_t o = sw128_offset(row, w);
            *reinterpret_cast<uint4 *>(xi + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(xi + kTile + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    } else {
        // gave up waiting: the copy and the MMAs already started complete before the CTA exits
        if (tid == 0) mbar_wait(&sm->full, 0, cx.limit);
        if (warp == 1 && lane == 0 && issued) mbar_wait(&sm->mma, 0, cx.limit);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 64);
    }
    // (a later part runs beside the chain before it; it has ended when both have)
    if (args.first > 0 && blockIdx.x == gridDim.x - 1) wait_for_last();
}

// ------------------------------------------------------------------ the chain
// Seven warpgroups: 0 to 3 own the state (warp w: TMEM lanes 32 (w % 4) .., quarter w / 4 of the tokens in steps 1 and 2 and of
// the state's rows in step 3), 4 (a lane quadrant per warp) brings V's columns to their lanes, 5 takes y from them to memory, and in
// 6 one warp issues the MMAs and one loads.  The two halves run staggered: the second one's products overlap the first one's
// conversions.
// Bound by the steps' latency: 2.2 us per chunk, of which the products 1 to 3 are 0.9 and the conversions between them the rest (143 us for
// the 64 chunks of B4 H16 T4096, whatever the heads' number up to one per SM; with 48 prompts of 128 to 8192 tokens and 16 heads, where
// all SMs have work, 0.19 of HBM's rate).  Code has to stay small here: fully unrolled it waited for instructions (5 us per chunk).
constexpr int kOwners = 16, kHelpers = 4, kBringer = 16, kTaker = 20, kIssuer = 24, kLoader = 25;
constexpr int kMThreads = 896;
constexpr int kGateRing = 4;
// registers per thread after the split (launched with 72): 4 x 80 + 48 + 88 + 48 = 7 x 72
constexpr int kRegsOwn = 80, kRegsBring = 48, kRegsTake = 88, kRegsRest = 48;
template <int KD>
struct ChainCfg {
    static constexpr uint32_t kTK = KD / 64 * kTile;    // a K or Q tile (64-feature blocks)
    // a stage (two): K, Q, V (two blocks of 64 columns), X's two parts, A
    static constexpr uint32_t kSK = 0, kSQ = kTK, kSV = 2 * kTK, kSX = kSV + 2 * kTile, kSA = kSX + 2 * kTile, kStage = kSA + kTile;
    static constexpr uint32_t kY = 2 * kStage;          // y of a chunk (4 KB per warp that takes it)
    static constexpr uint32_t kGates = kY + 2 * kTile;  // ring of kGateRing
    static constexpr uint32_t kSmall = kGates + kGateRing * 1024;
};
// TMEM columns (all 512 are allocated, so they start at 0): S^T (two parts); the accumulators P^T and E^T (then both dS^T),
// (Q S)^T, (A V')^T; R^T (two parts, then those of the decayed V'^T), V'^T, V^T
constexpr uint32_t kcS = 0, kcP = 128, kcE = 192, kcQS = 256, kcAV = 320, kcR = 384, kcW = 448, kcV = 480;

struct alignas(16) MSmall {
    uint64_t full_k[2], full_vx[2], full_qa[2];
    uint64_t got_s[2], got_r[2], got_w[2];   // an owner half's operand is in TMEM (4 warps)
    uint64_t got_v;                          // V^T is (the bringers)
    uint64_t y_read;                         // Q S and A V' have been read (the takers)
    uint64_t tail;                           // packed: the last chunk's rows of K past the end are 0 (the bringers)
    uint64_t done1[2], done2[2];             // halves of P, E
    uint64_t done2b;                         // the first half of R has been read
    // halves of dS of even and odd chunks, Q S and A V' (the loader may look at them late, but not two chunks late)
    uint64_t done3[4], done4[2];
    uint64_t fin;
    uint32_t tmem_base;
    int abort_flag;
};
#define MBAR(name, i) (sS + (uint32_t)offsetof(MSmall, name) + 8 * (uint32_t)(i))

template <int KD>
constexpr uint32_t kMSmemBytes = ChainCfg<KD>::kSmall + sizeof(MSmall) + 1024;
static_assert(kMSmemBytes<128> <= 232448, "shared memory budget");

template <int KD>
__global__ void __launch_bounds__(kMThreads, 1)
gdelta_chain_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const __grid_constant__ GdeltaTcArgs args)
{
    using Cfg = ChainCfg<KD>;
    constexpr int KH = KD / 2, KQ = KD / 4;     // half of the state's rows; an owner thread has a column, a quarter of its rows
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = align1024(smem_raw);
    MSmall *sm = reinterpret_cast<MSmall *>(base + Cfg::kSmall);
    const uint32_t s0 = smem_u32(base), sS = s0 + Cfg::kSmall;
    auto wait1 = [&](uint32_t bar, uint32_t parity) { return bounded_wait<false>(sS + offsetof(MSmall, abort_flag), bar, parity); };
    auto waitw = [&](uint32_t bar, uint32_t parity) { return bounded_wait<true>(sS + offsetof(MSmall, abort_flag), bar, parity); };

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = args.s.H, dv = args.s.dv;
    const bool packed = args.s.cu_seqlens != nullptr;
    const int tiles = (dv + 127) / 128;
    const int tile = blockIdx.x % tiles, h = blockIdx.x / tiles % H;
    int b = blockIdx.x / (tiles * H);
    Span sp;
    if (packed && !args.slot_base) {
        b = self_plan<false>(args, b, sp);
    } else {
        if (packed) {
            wait_for_last();
            b = args.order[b];
        }
        sp = span_of(args, b);
    }
    if (!sp.valid) return;
    const int c0 = args.first, T = sp.T - c0 * kC;      // tokens from this launch's first chunk on
    const int nch = args.chunks ? min(args.chunks, (T + kC - 1) / kC) : (T + kC - 1) / kC;
    const int ncols = min(128, dv - 128 * tile);        // of this CTA: 128 or 64
    const size_t bh = (size_t)b * H + h;
    const bool tail = packed && nch > 0 && T < nch * kC;

    if (tid == 0) {
        for (uint64_t *bar = sm->full_k; bar <= &sm->fin; ++bar)
            mbar_init(bar, bar >= sm->got_s && bar < &sm->got_v ? kOwners / 2 : bar >= &sm->got_v && bar <= &sm->tail ? kHelpers : 1);
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
    let_next_start();
    wait_for_last();

    if (warp >= kIssuer) {
        regs_dec<kRegsRest>();
        if (warp == kLoader && elect_one()) {
            const int hk = h / (H / args.s.Hk);
            const uint8_t *ws = args.ws + ((sp.slot + c0) * H + h) * kWsChunk;
            const size_t ws_step = (size_t)H * kWsChunk;      // from one chunk to the next
            auto tok = [&](uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int n, int heads, int head) {
                if (packed) tma_load(dst, map, bar, x, head, (int)sp.tok0 + n * kC);
                else tma_load(dst, map, bar, x, (c0 + n) * kC, b * heads + head);
            };
            int n1 = 0, n2 = 0;                    // chunks whose K, V, X / Q, A loads were started
            bool ok = true;
            // stage n & 1 takes chunk n once step 3 of chunk n - 2 has read K (and before it V, X and Q were read), and A V' after
            // it A
#pragma unroll 1
            for (int n = 0; n < nch && ok; ++n) {
                const uint32_t st = s0 + (n & 1) * Cfg::kStage, wph = ((n >> 1) - 1) & 1;
                const uint8_t *w = ws + n * ws_step;
                if (n >= 2) ok = wait1(MBAR(done3, 2 + (n & 1)), wph);
                if (!ok) break;
                uint32_t bar = MBAR(full_k, n & 1);
                bar_expect(bar, Cfg::kTK);
#pragma unroll 1
                for (int x = 0; x < KD / 64; ++x) tok(st + Cfg::kSK + x * kTile, &map_k, bar, 64 * x, n, args.s.Hk, hk);
                bar = MBAR(full_vx, n & 1);
                bar_expect(bar, ncols / 64 * kTile + 2 * kTile + kGateBytes);
                bulk_copy(s0 + Cfg::kGates + (n % kGateRing) * 1024, w + kWsGates, kGateBytes, bar);
#pragma unroll 1
                for (int x = 0; x < ncols / 64; ++x) tok(st + Cfg::kSV + x * kTile, &map_v, bar, 128 * tile + 64 * x, n, H, h);
                bulk_copy(st + Cfg::kSX, w + kWsX, 2 * kTile, bar);
                n1 = n + 1;
                if (n >= 2) ok = wait1(MBAR(done4, n & 1), wph);
                if (!ok) break;
                bar = MBAR(full_qa, n & 1);
                bar_expect(bar, Cfg::kTK + kTile);
#pragma unroll 1
                for (int x = 0; x < KD / 64; ++x) tok(st + Cfg::kSQ + x * kTile, &map_q, bar, 64 * x, n, args.s.Hk, hk);
                bulk_copy(st + Cfg::kSA, w + kWsA, kTile, bar);
                n2 = n + 1;
            }
            // loads still in flight complete before the CTA exits (also after a wait that was given up)
#pragma unroll 1
            for (int i = max(0, n1 - 2); i < n1; ++i) {
                wait1(MBAR(full_k, i & 1), (i >> 1) & 1);
                wait1(MBAR(full_vx, i & 1), (i >> 1) & 1);
                if (i < n2) wait1(MBAR(full_qa, i & 1), (i >> 1) & 1);
            }
        } else if (warp == kIssuer && elect_one()) {
            constexpr uint32_t id64 = idesc_bf16_f32(128, 64, false, false), id32 = idesc_bf16_f32(128, 32, false, false),
                               idS = idesc_bf16_f32(128, KH, false, true);
            constexpr uint32_t kHalfRows = (32 * 128) >> 4;       // from a tile's first 32 rows to its last
#pragma unroll 1
            for (int n = 0; n < nch; ++n) {
                const uint32_t st = s0 + (n & 1) * Cfg::kStage, ph = n & 1, fph = (n >> 1) & 1;
                const uint32_t klo = desc_lo(st + Cfg::kSK, 16), xlo = desc_lo(st + Cfg::kSX, 16);
                // 1  P^T = S^T K^T, both parts of S: the first half of S's rows for all tokens, the second one for one half
                // of the tokens after the other
                if (!wait1(MBAR(full_k, n & 1), fph)) break;
                if (tail && n == nch - 1 && !wait1(MBAR(tail, 0), 0)) break;
                if (!wait1(MBAR(got_s, 0), ph)) break;
                tc_fence_after();
#pragma unroll 4
                for (int i = 0; i < KD / 16; ++i) {        // part i % 2, k-step i / 2
                    const int kk = i >> 1;
                    mma_ts(kcP, kcS + (i & 1) * KH + kk * 8, klo + kk * 2, kHi128, id64, i > 0);
                }
                if (!wait1(MBAR(got_s, 1), ph)) break;
                tc_fence_after();
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    // (the second half of the rows: K's second block, or the second half of its one block's rows)
                    const uint32_t k2 = klo + t * kHalfRows + ((KD == 128 ? kTile : 64u) >> 4);
#pragma unroll 4
                    for (int i = 0; i < KD / 16; ++i) {
                        const int kk = i >> 1;
                        mma_ts(kcP + 32 * t, kcS + (i & 1) * KH + KD / 4 + kk * 8, k2 + kk * 2, kHi128, id32, true);
                    }
                    bar_commit(MBAR(done1, t));
                }
                // 2  E^T = R^T X^T: high X with both parts of R, low X with the high one.  X is lower triangular: the first
                // half of E needs the first half of R, the second one both.
                if (!wait1(MBAR(full_vx, n & 1), fph)) break;
                bool ok = true;
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    ok = wait1(MBAR(got_r, t), ph);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int o = t; o < 2; ++o) {          // half o of E from half t of R
                        const uint32_t d = kcE + 32 * o, xo = xlo + o * kHalfRows + 4 * t, r = kcR + 16 * t;
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk) {
                            mma_ts(d, r + kk * 8, xo + kk * 2, kHi128, id32, t + kk > 0);
                            mma_ts(d, r + 32 + kk * 8, xo + kk * 2, kHi128, id32, true);
                            mma_ts(d, r + kk * 8, xo + kk * 2 + (kTile >> 4), kHi128, id32, true);
                        }
                        if (t + o == 0) bar_commit(MBAR(done2, 0));
                    }
                    bar_commit(t == 0 ? MBAR(done2b, 0) : MBAR(done2, 1));
                }
                if (!ok) break;
                // (Q S)^T
                if (!wait1(MBAR(full_qa, n & 1), fph) || (n > 0 && !wait1(MBAR(y_read, 0), ph ^ 1))) break;
                tc_fence_after();
                const uint32_t qlo = desc_lo(st + Cfg::kSQ, 16), alo = desc_lo(st + Cfg::kSA, 16);
#pragma unroll 4
                for (int kk = 0; kk < KD / 16; ++kk)
                    mma_ts(kcQS, kcS + kk * 8, qlo + (kk >> 2) * (kTile >> 4) + (kk & 3) * 2, kHi128, id64, kk > 0);
                // 3  dS^T = V'^T K, both parts of the decayed V', one half of the state's rows after the other
                if (!wait1(MBAR(got_w, 0), ph) || !wait1(MBAR(got_w, 1), ph)) break;
                tc_fence_after();
                const uint32_t kmn = desc_lo(st + Cfg::kSK, kTile);
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    const uint32_t ko = kmn + t * ((KD == 128 ? kTile : 64u) >> 4);
#pragma unroll 4
                    for (int i = 0; i < 8; ++i) {          // part i / 4, k-step i % 4
                        const int kk = i & 3;
                        mma_ts(kcP + 64 * t, kcR + (i >> 2) * 32 + kk * 8, ko + kk * (2048 >> 4), kHi128, idS, i > 0);
                    }
                    bar_commit(MBAR(done3, 2 * t + (n & 1)));
                }
                // (A V')^T
#pragma unroll 4
                for (int kk = 0; kk < 4; ++kk) mma_ts(kcAV, kcW + kk * 8, alo + kk * 2, kHi128, id64, kk > 0);
                bar_commit(MBAR(done4, n & 1));
            }
            // every MMA completes before the CTA exits
            bar_commit(MBAR(fin, 0));
            wait1(MBAR(fin, 0), 0);
        }
        __syncwarp();
    } else if (warp >= kTaker) {
        regs_inc<kRegsTake>();
        const int q4 = warp & 3;
        const uint32_t tq = (uint32_t)(32 * q4) << 16;
        const uint32_t buf = s0 + Cfg::kY + 4096 * q4;
        const size_t y_step = (packed ? (size_t)H : 1) * dv;
        // this lane's column and token of a block of 8 when rows go out
        const int out_col = 32 * q4 + 8 * (lane & 3), out_tok = lane >> 2;
        uint16_t *const y0 = args.y + (packed ? (sp.tok0 * H + h) * dv : (bh * args.s.T + (size_t)c0 * kC) * dv) + 128 * tile + out_col + (size_t)out_tok * y_step;
        const float2 scale = make_float2(args.scale, args.scale);
#pragma unroll 1
        for (int n = 0; n < nch; ++n) {
            // y, by way of shared memory to whole rows (the gates have been waited for by those whose products this waits for)
            if (!waitw(MBAR(done4, n & 1), (n >> 1) & 1)) break;
            tc_fence_after();
            const uint32_t eg = s0 + Cfg::kGates + (n % kGateRing) * 1024;
#pragma unroll 1
            for (int x = 0; x < 4; ++x) {
                float qs[16], av[16];
                tc_ld_32x32b_x16(tq + kcQS + 16 * x, qs);
                tc_ld_32x32b_x16(tq + kcAV + 16 * x, av);
                wait_loaded(qs);
                wait_loaded(av);
                if (x == 3) {
                    tc_fence_before();
                    bar_arrive_warp(MBAR(y_read, 0));
                }
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 g = lds_f4(eg + 64 * x + 16 * i);
                    const float2 y01 = __fmul2_rn(scale, __ffma2_rn(make_float2(g.x, g.y), make_float2(qs[4 * i], qs[4 * i + 1]),
                                                                   make_float2(av[4 * i], av[4 * i + 1])));
                    const float2 y23 = __fmul2_rn(scale, __ffma2_rn(make_float2(g.z, g.w), make_float2(qs[4 * i + 2], qs[4 * i + 3]),
                                                                   make_float2(av[4 * i + 2], av[4 * i + 3])));
                    w[2 * i] = pack_bf16x2(y01.x, y01.y);
                    w[2 * i + 1] = pack_bf16x2(y23.x, y23.y);
                }
                cols_put(buf, lane, 2 * x, w[0], w[1], w[2], w[3]);
                cols_put(buf, lane, 2 * x + 1, w[4], w[5], w[6], w[7]);
            }
            __syncwarp();
            const int rows = T - n * kC - out_tok;
            uint16_t *yp = y0 + (size_t)(n * kC) * y_step;
#pragma unroll 2
            for (int w = 0; w < 8; ++w) {
                const uint4 v = cols_get(buf, lane, w);
                if (8 * w < rows && out_col < ncols) *reinterpret_cast<uint4 *>(yp + (size_t)(8 * w) * y_step) = v;
            }
            __syncwarp();
        }
        tc_fence_before();
    } else if (warp >= kBringer) {
        regs_dec<kRegsBring>();
        const int q4 = warp & 3, d = 32 * q4 + lane;    // lane quadrant, value column of the CTA
        const uint32_t tq = (uint32_t)(32 * q4) << 16;
        const uint32_t c16 = (d & 63) >> 3, col = (d >> 6) * kTile + (d & 7) * 2;   // this column in a tile of V
#pragma unroll 1
        for (int n = 0; n < nch; ++n) {
            // this thread's column of V (0 past the sequence's end), once the owners have read the last chunk's
            const uint32_t st = s0 + (n & 1) * Cfg::kStage;
            if (!waitw(MBAR(full_vx, n & 1), (n >> 1) & 1)) break;
            if (n > 0 && !(waitw(MBAR(got_r, 0), (n - 1) & 1) && waitw(MBAR(got_r, 1), (n - 1) & 1))) break;
            const int left = T - n * kC;
            if (tail && n == nch - 1) {
                // rows of K past the end hold another sequence's keys, which step 3 would multiply by 0: they become 0
                if (!waitw(MBAR(full_k, n & 1), (n >> 1) & 1)) break;
                for (int x = tid - 32 * kBringer; x < (kC - left) * (KD / 8); x += 32 * kHelpers) {
                    const int c = x % (KD / 8);
                    sts4(st + Cfg::kSK + (c >> 3) * kTile + sw128_offset(left + x / (KD / 8), c & 7), 0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                bar_arrive_warp(MBAR(tail, 0));
            }
            tc_fence_after();
            const int last = d < ncols ? left : 0;
#pragma unroll 1
            for (int x = 0; x < 4; ++x) {
                uint32_t v[8];
                const uint32_t a = st + Cfg::kSV + col + x * (16 * 128);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int t = 2 * i;
                    const uint32_t lo = lds_u16(a + t * 128 + ((c16 ^ (t & 7)) << 4)),
                                   hi = lds_u16(a + (t + 1) * 128 + ((c16 ^ ((t + 1) & 7)) << 4));
                    v[i] = (16 * x + t < last ? lo : 0) | (16 * x + t + 1 < last ? hi << 16 : 0);
                }
                tm_st8(tq + kcV + 8 * x, v);
            }
            tc_wait_st();
            tc_fence_before();
            bar_arrive_warp(MBAR(got_v, 0));
        }
        tc_fence_before();
    } else {
        regs_inc<kRegsOwn>();
        const int q4 = warp & 3, cq = warp >> 2, ch = cq >> 1, d = 32 * q4 + lane;
        const uint32_t tq = (uint32_t)(32 * q4) << 16;
        const bool live = d < ncols;
        float2 S[KQ / 2];                               // S[i]: state rows KQ cq + 2 i, + 1 of the lane's column
        const size_t s_at = (bh * KD + KQ * cq) * dv + 128 * tile + d;
#pragma unroll
        for (int i = 0; i < KQ / 2; ++i) {
            S[i] = make_float2(0.f, 0.f);
            if (args.S0 && live) S[i] = make_float2(__ldcg(args.S0 + s_at + (size_t)(2 * i) * dv), __ldcg(args.S0 + s_at + (size_t)(2 * i + 1) * dv));
        }
        // rows 16 x .. of this quarter as left operands
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
        if (nch > 0) {
#pragma unroll
            for (int x = 0; x < KQ / 16; ++x) put_s(x, S + 8 * x);
            stored(MBAR(got_s, ch));
        }
        bool ok = true;
#pragma unroll 1
        for (int n = 0; n < nch; ++n) {
            const uint32_t ph = n & 1, gates = s0 + Cfg::kGates + (n % kGateRing) * 1024 + 64 * cq;
            // R^T = V^T - e^G P^T, tokens 16 cq ..  (past the sequence's end V and P are 0)
            ok = waitw(MBAR(full_vx, n & 1), (n >> 1) & 1) && waitw(MBAR(got_v, 0), ph) && waitw(MBAR(done1, ch), ph);
            if (!ok) break;
            tc_fence_after();
            {
                float p[16], v[8];
                tc_ld_32x32b_x16(tq + kcP + 16 * cq, p);
                tm_ld8(tq + kcV + 8 * cq, v);
                wait_loaded(p);
                wait_loaded(v);
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 g = lds_f4(gates + 16 * i);
                    const uint32_t v0 = __float_as_uint(v[2 * i]), v1 = __float_as_uint(v[2 * i + 1]);
                    split(__ffma2_rn(make_float2(-g.x, -g.y), make_float2(p[4 * i], p[4 * i + 1]), make_float2(bf16_lo(v0), bf16_hi(v0))),
                          hi[2 * i], lo[2 * i]);
                    split(__ffma2_rn(make_float2(-g.z, -g.w), make_float2(p[4 * i + 2], p[4 * i + 3]), make_float2(bf16_lo(v1), bf16_hi(v1))),
                          hi[2 * i + 1], lo[2 * i + 1]);
                }
                tm_st8(tq + kcR + 8 * cq, hi);
                tm_st8(tq + kcR + 32 + 8 * cq, lo);
            }
            stored(MBAR(got_r, ch));
            // V'^T = beta E^T, and decayed to the chunk's end
            ok = waitw(MBAR(done2, ch), ph);
            if (!ok) break;
            tc_fence_after();
            {
                float e[16];
                tc_ld_32x32b_x16(tq + kcE + 16 * cq, e);
                wait_loaded(e);
                uint32_t w[8], hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 er = lds_f4(gates + 4 * kC + 16 * i), be = lds_f4(gates + 8 * kC + 16 * i);
                    const float2 w0 = __fmul2_rn(make_float2(be.x, be.y), make_float2(e[4 * i], e[4 * i + 1]));
                    const float2 w1 = __fmul2_rn(make_float2(be.z, be.w), make_float2(e[4 * i + 2], e[4 * i + 3]));
                    w[2 * i] = pack_bf16x2(w0.x, w0.y);
                    w[2 * i + 1] = pack_bf16x2(w1.x, w1.y);
                    split(__fmul2_rn(make_float2(er.x, er.y), w0), hi[2 * i], lo[2 * i]);
                    split(__fmul2_rn(make_float2(er.z, er.w), w1), hi[2 * i + 1], lo[2 * i + 1]);
                }
                tm_st8(tq + kcW + 8 * cq, w);
                // (the second half of E has read the first one's R)
                ok = ch || waitw(MBAR(done2b, 0), ph);
                if (!ok) break;
                tc_fence_after();
                tm_st8(tq + kcR + 8 * cq, hi);
                tm_st8(tq + kcR + 32 + 8 * cq, lo);
            }
            stored(MBAR(got_w, ch));
            const float gC = ldsf(gates - 64 * cq + 4 * (kC - 1));
            ok = waitw(MBAR(done3, 2 * ch + (n & 1)), (n >> 1) & 1);
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
                if (n + 1 < nch) put_s(x, S + 8 * x);
            }
            if (n + 1 < nch) stored(MBAR(got_s, ch));
        }
        if (ok && live) {
#pragma unroll
            for (int i = 0; i < KQ / 2; ++i) {
                args.S_out[s_at + (size_t)(2 * i) * dv] = S[i].x;
                args.S_out[s_at + (size_t)(2 * i + 1) * dv] = S[i].y;
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

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

}  // namespace

long long gdelta_tc_slots(int B, int T, bool packed)
{
    return packed ? (long long)T / kC + B : (long long)B * ((T + kC - 1) / kC);
}

size_t gdelta_tc_plan_bytes(int B) { return round_up((2 * (size_t)B + 1) * sizeof(int), 256); }

size_t gdelta_tc_workspace_bytes(int B, int H, int T, bool packed)
{
    return (packed ? gdelta_tc_plan_bytes(B) : 0) + (size_t)gdelta_tc_slots(B, T, packed) * H * kWsChunk;
}

template <int KD, bool BACK>
static cudaError_t launch_prep(const CUtensorMap &q, const CUtensorMap &k, const GdeltaTcArgs &a, cudaStream_t stream)
{
    static OncePerDevice once;
    const cudaError_t e = set_smem_once(gdelta_prep_kernel<KD, BACK>, kPSmemBytes, once);
    if (e != cudaSuccess) return e;
    const long long n = (a.chunks ? (long long)a.s.B * a.chunks : gdelta_tc_slots(a.s.B, a.s.T, a.s.cu_seqlens != nullptr)) * a.s.H;
    if (n > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (n == 0) return cudaSuccess;
    // (after the plan; a later part: beside the chain before it; else nothing to start ahead of)
    if (a.slot_base || a.first) return launch_after(gdelta_prep_kernel<KD, BACK>, (unsigned)n, kPThreads, kPSmemBytes, stream, q, k, a);
    gdelta_prep_kernel<KD, BACK><<<(unsigned)n, kPThreads, kPSmemBytes, stream>>>(q, k, a);
    return cudaGetLastError();
}

cudaError_t launch_gdelta_prep_backward(const CUtensorMap &q, const CUtensorMap &k, const GdeltaTcArgs &a, cudaStream_t stream)
{
    return a.s.r == 64 ? launch_prep<64, true>(q, k, a, stream) : launch_prep<128, true>(q, k, a, stream);
}

template <int KD>
static cudaError_t launch_as(const GdeltaTcMaps &m, const GdeltaTcArgs &a, int sms, cudaStream_t stream)
{
    static OncePerDevice once_m;
    cudaError_t e = set_smem_once(gdelta_chain_kernel<KD>, kMSmemBytes<KD>, once_m);
    if (e != cudaSuccess) return e;
    const GdeltaShape &s = a.s;
    const long long nmain = (long long)s.B * s.H * ((s.dv + 127) / 128);
    if (nmain > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (a.slot_base) {
        gdelta_plan_kernel<<<1, kPlanThreads, 0, stream>>>(s.cu_seqlens, s.B, s.T, a.slot_base, a.order, s.status);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    // Few heads leave SMs without a chain: there the sequences go in two parts, and the second one's A and X are formed beside the
    // chain of the first.  The first part is a little less than what that chain gives time for (3 of 10 chunks: B4 H16 T4096
    // 200 -> 188 us, T16384 749 -> 703, B1 H16 T16384 611 -> 585; 45 of 100 194, 20 194, three parts 191).  Another launch of the chain costs
    // about 5 us, which fewer than 8 chunks per SM do not repay.
    GdeltaTcArgs part = a;
    const int nch = (s.T + kC - 1) / kC;
    const bool apart = !s.cu_seqlens && 2 * nmain <= sms && (long long)s.B * s.H * nch >= 8LL * sms && nch >= 16;
    if (apart) part.chunks = (int)(nch * 3LL / 10);
    for (;;) {
        if ((e = launch_prep<KD, false>(m.q, m.k, part, stream)) != cudaSuccess) return e;
        e = launch_after(gdelta_chain_kernel<KD>, (unsigned)nmain, kMThreads, kMSmemBytes<KD>, stream, m.q, m.k, m.v, part);
        if (e != cudaSuccess || !apart || part.first) return e;
        part.first = part.chunks, part.chunks = nch - part.first;
        part.S0 = a.S_out;
    }
}

cudaError_t launch_gdelta_tc(const GdeltaTcMaps &m, const GdeltaTcArgs &a, int sms, cudaStream_t stream)
{
    GdeltaTcArgs self = a;
    if (a.s.B <= kSelfPlan) self.slot_base = self.order = nullptr;
    return a.s.r == 64 ? launch_as<64>(m, self, sms, stream) : launch_as<128>(m, self, sms, stream);
}

}  // namespace la
