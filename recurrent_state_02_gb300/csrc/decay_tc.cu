// decay_tc.cu -- the decayed linear attention's sweep in chunks on the sm_103a tensor
// cores (tcgen05 MMAs, TMEM accumulators, TMA tiles), for BF16.
//
// A sweep (decay.h) over a chunk of n <= C = 128 tokens whose entering state is S, with the
// token at row i in position p_i of the sweep's own order (p_i = i forwards, n-1-i
// backwards) and late = backwards:
//     out_i = s_in sum_{p_j <= p_i} g^{p_i - p_j} (a_i . b_j) c_j  +  s_out g^{p_i + 1 - late} a_i^T S
//     S'    = g^n S + sum_j w g^{n - 1 + late - p_j} b_j c_j^T
// (s_out the output scale, w the write scale, s_in = s_out w).  As matrices:
//     P   = A B^T                    M=128 N=128 K=ra   -> TMEM
//     P   <- P . g^{p_i - p_j}       in registers, masked, back to TMEM as BF16
//     Yi  = P C                      M=128 N=64  K=128  (P from TMEM)
//     Ye  = A S                      M=128 N=64  K=ra   (S as BF16)
//     dS  = B^T [Ch | Cl]            M=ra  N=128 K=128  (Ch + Cl = diag(w g^..) C in two BF16 parts)
// and out = s_in Yi + s_out g^.. Ye leaves through a TMA store from the chunk's tile of
// C, which is done with by then.
//
// The state is FP32 in the registers of four warps: after each chunk S <- g^n S + dS
// (both halves), so that its rounding is that of one FP32 sum per chunk.  Two
// BF16 parts of the weighted values keep the state to 2^-16 per term, where one
// part would leave 2^-8; the outputs, which are BF16, take P and S rounded once.  (A third part leaves
// FP32's own rounding, 1.7e-7 of the state's norm in place of 2.4e-6, but its tile takes the place of a quarter
// of a's buffers: 62.5 us at B4 H16 T4096 against 55.6.  The same prompt as FP32 takes the FP32 recurrence.)
//
// No power of g is ever divided by: a block of 32 x 32 scores below the diagonal carries
// g^{p_i - p_j} as the product of a row's power and a column's power, both with
// exponents >= 0; a diagonal block looks its powers up.  So every g in 0 .. 1 (0 too)
// takes the same path, and what underflows is negligible next to the diagonal.
//
// One CTA owns one (b, h, 64 columns of c) and walks its chunks, or, where that leaves
// most SMs idle, one segment of them: a state pass then forms what every part of the
// sweep adds to the state ("门控递推为什么能做并行 scan？" of "Linear attention：把历史写进状态":
// updates compose as affine maps, and with a constant decay the map of a part is
// g^tokens and that sum), and a later segment starts from the parts before it.
//
// Four warpgroups (each of a group's warps reaches the TMEM lanes of its quadrant): TMA
// producer and three MMA issuers (scores, dS, outputs, so that none waits for another's
// operands); scores; weighted values; state and outputs.  The groups run different code
// at the same time, and what they run has to fit the instruction cache: with every loop
// unrolled and long waits the same arithmetic took 238 us where it now takes 55.
//
// Bound by shared memory: counting one read of each operand per MMA, a chunk moves about
// 370 KB through it (P 64, Ye 48, Yi 16, dS 64, loads 80, stores 16, the weighted values
// 48, state and outputs 32), 2900 cycles at 128 bytes a cycle, or 1.5 us of the 1.6 that it takes; at
// HBM's rate it would be 1.3.  Measured at r = dv = 128: B4 H16 T4096 55 us (272 MB, 74 % of the copy
// bandwidth), B1 H32 T65536 in segments 529 us, the gradients' three sweeps of
// B4 H16 T4096 162 us.
#include "decay.h"
#include "tc_short.cuh"

#include <cstddef>

namespace la {
namespace {

constexpr int kCT = 128;                       // tokens per chunk
constexpr int kThreads = 512;
// registers per thread after the split (launched with 128): 56 + 128 + 120 + 208 = 4 * 128
constexpr int kRegsIssue = 56, kRegsValues = 120, kRegsState = 208;
constexpr uint32_t kBlk = kCT * 128;           // 16 KB: 128 rows x 64 BF16 columns, 128-byte swizzle
constexpr int kStC = 3;                        // stages of c (a and b have two)

// Packed batches of at most this many sequences run the longest first.
constexpr int kOrdered = 256;

// TMEM columns
constexpr uint32_t kColP = 0, kColYi = 256, kColYe = 320, kColDS = 384;

template <int KD>
struct Lay {
    static constexpr int NB = KD / 64;                       // 64-column blocks of a and b
    static constexpr uint32_t kTile = NB * kBlk;
    static constexpr uint32_t kOffA = 0, kOffB = 2 * kTile, kOffC = 4 * kTile;
    static constexpr uint32_t kOffW = kOffC + kStC * kBlk;   // weighted values: Ch, Cl
    static constexpr uint32_t kOffS = kOffW + 2 * kBlk;      // the state as BF16 [128 x 64] (KD rows are read)
    static constexpr uint32_t kOffSmall = kOffS + kBlk;
};

struct alignas(16) SmallD {
    uint64_t fullA[2], fullB[2], fullC[kStC], emptyA[2], emptyB[2], emptyC[kStC];
    uint64_t p_raw[2], p_ready[2], p_free[2], w_full, w_empty, ds_full, ds_empty, s_full, ye_full, yi_full, yi_empty, tail, done[3];
    uint32_t tmem_base;
    int abort_flag;
    alignas(16) float pw[kCT + 4];     // g^0 .. g^128
    float gpart;                       // g^(tokens of a part)
    int seq[3];                        // packed: this CTA's sequence and its bounds
    int len[kOrdered];                 // and the lengths of all
};

// shared-memory address of a barrier (in the kernel: sS is the SmallD's)
#define BAR(name, i) (sS + (uint32_t)offsetof(SmallD, name) + 8 * (uint32_t)(i))

template <int KD>
constexpr uint32_t smem_bytes() { return Lay<KD>::kOffSmall + sizeof(SmallD) + 1024; }
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory budget");

// PACKED: packed sequences (forwards); REV: the launch has backward sweeps (of [B,H,T,d] arrays).
// STATE: the state pass of a split sweep: what each part of it adds to the state, from zero; only b and
// c are read, only dS is formed.
template <int KD, bool PACKED, bool REV, bool STATE>
__global__ void __launch_bounds__(kThreads, 1)
decay_tc_kernel(const __grid_constant__ DecayTcParams args)
{
    using L = Lay<KD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    SmallD *sm = reinterpret_cast<SmallD *>(base + L::kOffSmall);
    const uint32_t s0 = smem_u32(base), sS = s0 + L::kOffSmall;
    auto wait1 = [&](uint32_t bar, uint32_t parity) { return bounded_wait<false>(sS + offsetof(SmallD, abort_flag), bar, parity); };
    auto waitw = [&](uint32_t bar, uint32_t parity) { return bounded_wait<true>(sS + offsetof(SmallD, abort_flag), bar, parity); };
    auto power = [&](int e) { return ldsf(sS + (uint32_t)offsetof(SmallD, pw) + 4 * e); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    int tile = blockIdx.x, which = 0;
    while (tile >= args.tiles[which]) tile -= args.tiles[which++];
    const DecaySweep &sw = args.sw[which];
    const TcSweepMaps &maps = args.maps[which];
    const int h = blockIdx.y, H = args.d.H, n_all = sw.n, c0 = tile * 64;
    constexpr bool packed = PACKED;
    const bool rev = REV && sw.rev;

    // this CTA's sequence
    const int B = args.B, z = blockIdx.z / B;      // z: the segment, or part, of the sweep
    int b = blockIdx.z % B, T = args.d.T, seq0 = 0;
    if (packed) {
        int seq1 = 0;
        if (B <= kOrdered) {
            // CTA row z takes the sequence with z longer ones (equal ones in order), so that no long one starts last.
            // H = 16: a prompt of 16384 tokens behind 47 of 512, 323 us in the batch's own order, 215 so;
            // 48 prompts of 128 .. 8192 tokens, 343 and 350.
            int start = 0;
            if (tid < B) {
                start = args.d.cu_seqlens[tid];
                sm->len[tid] = args.d.cu_seqlens[tid + 1] - start;
            }
            __syncthreads();
            if (tid < B) {
                const int mine = sm->len[tid];
                int rank = 0;
#pragma unroll 8
                for (int i = 0; i < B; ++i) {
                    const int other = sm->len[i];
                    rank += other > mine || (other == mine && i < tid);
                }
                if (rank == b) sm->seq[0] = tid, sm->seq[1] = start, sm->seq[2] = start + mine;
            }
            __syncthreads();
            b = sm->seq[0], seq0 = sm->seq[1], seq1 = sm->seq[2];
        } else {
            seq0 = args.d.cu_seqlens[b];
            seq1 = args.d.cu_seqlens[b + 1];
        }
        // (bad bounds are recorded by the token kernel's launch, which looks at every sequence)
        if (seq0 < 0 || seq1 < seq0 || seq1 > args.d.T) return;
        T = seq1 - seq0;
        if (T < args.d.len_min || T > args.d.len_max) return;
    }
    const size_t bh = (size_t)b * H + h;
    // the chunks of the sweep, and the run of them that is this CTA's: all, a segment or a part
    const int all = (T + kCT - 1) / kCT, run = STATE ? args.part_chunks : args.seg_chunks;
    const int cb = packed ? 0 : z * run, nch = packed || run == 0 ? all : min(run, all - cb);
    // chunk of this CTA's step c, its first token and its tokens
    auto chunk_t0 = [&](int c) { return (rev ? all - 1 - cb - c : cb + c) * kCT; };
    auto chunk_n = [&](int c) { return min(kCT, T - chunk_t0(c)); };

    // Loads of a chunk, by thread 0: its boxes in the order in which their buffers come free: b and a of
    // chunk c after chunk c - 2's dS and Ye, c once chunk c - 3's outputs have left.  Each is followed by an
    // L2 prefetch of the same box two chunks on, whose buffer is still in use (a, b: by the
    // head's first tile only, the others read the same).
    constexpr uint32_t kHi = desc_hi(1024, 2);
    const uint32_t sA = s0 + L::kOffA, sB = s0 + L::kOffB, sC = s0 + L::kOffC;
    int loaded = 0;
    auto load_chunk = [&](int c) -> bool {
        const int s = c & 1, t0 = chunk_t0(c), t2 = chunk_t0(c + 2);
#pragma unroll 1
        for (int i = 0; i <= 2 * L::NB; ++i) {
            if (STATE && i >= L::NB && i < 2 * L::NB) continue;
            const bool is_c = i == 2 * L::NB, is_a = i >= L::NB;
            const int k = is_c ? 0 : is_a ? i - L::NB : i, x = is_c ? c0 : 64 * k;
            const uint32_t full = is_c ? BAR(fullC, c % kStC) : is_a ? BAR(fullA, s) : BAR(fullB, s);
            const uint32_t dst = is_c ? sC + (c % kStC) * kBlk : (is_a ? sA : sB) + s * L::kTile + k * kBlk;
            const CUtensorMap *map = is_c ? &maps.c : is_a ? &maps.a : &maps.b;
            if (k == 0) {
                const uint32_t empty = is_c ? BAR(emptyC, c % kStC) : is_a ? BAR(emptyA, s) : BAR(emptyB, s);
                if (c >= (is_c ? kStC : 2) && !wait1(empty, (is_c ? c / kStC - 1 : (c >> 1) - 1) & 1)) return false;
                bar_expect(full, is_c ? kBlk : L::kTile);
            }
            tma_load(dst, map, full, x, packed ? h : t0, packed ? seq0 + t0 : (int)bh);
            if (c + 2 < nch && (is_c || tile == 0)) tma_prefetch_l2_3d(map, x, packed ? h : t2, packed ? seq0 + t2 : (int)bh);
            loaded = c * 3 + (is_c ? 3 : is_a ? 2 : 1);
        }
        return true;
    };

    // ------------------------------------------------------------ set-up
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm->fullA[s], 1);
            mbar_init(&sm->fullB[s], 1);
            mbar_init(&sm->emptyA[s], 2);      // read by the scores and by Ye
            mbar_init(&sm->emptyB[s], STATE ? 1 : 2);      // read by the scores and by dS
            mbar_init(&sm->p_raw[s], 1);
            mbar_init(&sm->p_ready[s], 4);
            mbar_init(&sm->p_free[s], 1);
        }
        for (int s = 0; s < kStC; ++s) {
            mbar_init(&sm->fullC[s], 1);
            mbar_init(&sm->emptyC[s], 4);      // the output rows of four warps have left it
        }
        mbar_init(&sm->w_full, 4);
        mbar_init(&sm->w_empty, 1);
        mbar_init(&sm->ds_full, 1);
        mbar_init(&sm->ds_empty, 4);
        mbar_init(&sm->s_full, 4);
        mbar_init(&sm->ye_full, 1);
        mbar_init(&sm->yi_full, 1);
        mbar_init(&sm->yi_empty, 4);
        mbar_init(&sm->tail, 4);
        for (int i = 0; i < 3; ++i) mbar_init(&sm->done[i], 1);
        sm->abort_flag = 0;
        fence_mbarrier_init();
        if (nch > 0) load_chunk(0);     // in flight during the rest of the set-up
        tma_prefetch_desc(&maps.out);
    }
    if (warp == 1) {
        tmem_alloc(&sm->tmem_base, 512);
        tmem_relinquish();
    }
    if (tid >= 128 && tid - 128 <= kCT) {
        // powers of g from its repeated squares in 64 bits: each entry is rounded once
        const int e = tid - 128;
        double p = 1.0, q = (double)args.d.decay[h];
        for (int bit = 0; bit < 8; ++bit) {
            if (e >> bit & 1) p *= q;
            q *= q;
        }
        sm->pw[e] = (float)p;
        if (e == 0 && !STATE) {
            // what a part of a split sweep decays an entering state by (all are full but the first of a
            // backward sweep, which nothing enters)
            double r = 1.0, x = (double)args.d.decay[h];
            for (long long n = z > 1 || args.nparts > 1 ? (long long)args.part_chunks * kCT : 0; n; n >>= 1, x *= x)
                if (n & 1) r *= x;
            sm->gpart = (float)r;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm->tmem_base;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int row = (warp & 3) * 32 + lane;     // the TMEM lane, and tile row, of this thread
    const int group = warp >> 2;

    if (group == 0) {
        regs_dec<kRegsIssue>();
        if (warp == 0 && lane == 0) {
            // --------------------------------------------------- producer
            for (int c = 1; c < nch && load_chunk(c); ++c) {}
            // every issued load lands before the CTA may exit (those of the last three chunks, in order)
            for (int i = max(0, loaded - 9); i < loaded; ++i) {
                const int c = i / 3, k = i % 3;
                if (STATE && k == 1) continue;
                if (k == 2) wait1(BAR(fullC, c % kStC), (c / kStC) & 1);
                else if (3 * (c + 2) + k >= loaded) wait1(k ? BAR(fullA, c & 1) : BAR(fullB, c & 1), (c >> 1) & 1);
            }
        } else if (!STATE && warp == 1 && lane == 0) {
            // ------------------------------------------------- MMA: scores
            constexpr uint32_t idP = idesc_bf16_f32(128, 128, false, false);
            for (int c = 0; c < nch; ++c) {
                const int s = c & 1;
                if (!wait1(BAR(fullB, s), (c >> 1) & 1) || !wait1(BAR(fullA, s), (c >> 1) & 1)) break;
                // the rows behind a packed sequence (in its last chunk) become zeros in b and c before its scores, and
                // so its Yi, are formed: what lies there may be anything, and a mask of zeros would let it through.
                // A barrier of one phase: one that every chunk completes would have to be waited for in
                // every chunk, as a wait by parity also returns when the phase before is still open.
                if (packed && c == nch - 1 && chunk_n(c) < kCT && !wait1(BAR(tail, 0), 0)) break;
                // the buffer held P of chunk c - 2, whose product is done
                if (c >= 2 && !wait1(BAR(p_free, s), ((c >> 1) - 1) & 1)) break;
                tc_fence_after();
                const uint32_t alo = desc_lo(sA + s * L::kTile, 16), blo = desc_lo(sB + s * L::kTile, 16);
                const uint32_t d = tmem + kColP + s * 128;
#pragma unroll 1
                for (int k = 0; k < KD / 16; ++k) {
                    const uint32_t o = ((k >> 2) * kBlk + (k & 3) * 32) >> 4;
                    mma_ss(d, alo + o, kHi, blo + o, kHi, idP, k > 0);
                }
                bar_commit(BAR(p_raw, s));
                bar_commit(BAR(emptyA, s));
                bar_commit(BAR(emptyB, s));
            }
        } else if (warp == 2 && lane == 0) {
            // ----------------------------------------------------- MMA: dS
            constexpr uint32_t idDS = idesc_bf16_f32(128, 128, true, true);
            for (int c = 0; c < nch; ++c) {
                const int s = c & 1;
                if (!wait1(BAR(fullB, s), (c >> 1) & 1) || !wait1(BAR(w_full, 0), c & 1)) break;
                if (c >= 1 && !wait1(BAR(ds_empty, 0), (c - 1) & 1)) break;
                tc_fence_after();
                // (ra = 64: rows 64 .. 127 of the product come from the tile behind b and are not used)
                const uint32_t alo = desc_lo(sB + s * L::kTile, kBlk), blo = desc_lo(s0 + L::kOffW, kBlk);
#pragma unroll 1
                for (int k = 0; k < 8; ++k) {
                    const uint32_t o = k * (2048 >> 4);
                    mma_ss(tmem + kColDS, alo + o, kHi, blo + o, kHi, idDS, k > 0);
                }
                bar_commit(BAR(ds_full, 0));
                bar_commit(BAR(w_empty, 0));
                bar_commit(BAR(emptyB, s));
            }
        } else if (!STATE && warp == 3 && lane == 0) {
            // ------------------------------------------------ MMA: outputs
            constexpr uint32_t idY = idesc_bf16_f32(128, 64, false, true);
            for (int c = 0; c < nch; ++c) {
                const int s = c & 1;
                // (the state of chunk c is published once Ye of chunk c - 1 has been read)
                if (!wait1(BAR(fullA, s), (c >> 1) & 1) || !wait1(BAR(s_full, 0), c & 1)) break;
                tc_fence_after();
                {
                    const uint32_t alo = desc_lo(sA + s * L::kTile, 16), blo = desc_lo(s0 + L::kOffS, kBlk);
#pragma unroll 1
                    for (int k = 0; k < KD / 16; ++k) {
                        const uint32_t o = ((k >> 2) * kBlk + (k & 3) * 32) >> 4;
                        mma_ss(tmem + kColYe, alo + o, kHi, blo + k * (2048 >> 4), kHi, idY, k > 0);
                    }
                }
                bar_commit(BAR(ye_full, 0));
                bar_commit(BAR(emptyA, s));
                if (!wait1(BAR(fullC, c % kStC), (c / kStC) & 1) || !wait1(BAR(p_ready, s), (c >> 1) & 1)) break;
                if (c >= 1 && !wait1(BAR(yi_empty, 0), (c - 1) & 1)) break;
                tc_fence_after();
                const uint32_t blo = desc_lo(sC + (c % kStC) * kBlk, kBlk), a = tmem + kColP + s * 128;
#pragma unroll 1
                for (int k = 0; k < 8; ++k) mma_ts(tmem + kColYi, a + 8 * k, blo + k * (2048 >> 4), kHi, idY, k > 0);
                bar_commit(BAR(yi_full, 0));
                bar_commit(BAR(p_free, s));
            }
        }
        if (warp >= 1 && lane == 0) {
            // every MMA that this thread issued completes before TMEM is released
            bar_commit(BAR(done, warp - 1));
            wait1(BAR(done, warp - 1), 0);
        }
        __syncwarp();
    } else if (group == 1) {
        // --------------------------------------------------------- scores
        // the powers of a diagonal block's row (0 behind the mask), and of a column of the blocks below: the same
        // for every chunk
        const int R = warp & 3;
        float2 wd[16], wc[16];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const int e = rev ? j - lane : lane - j;
            const float d = power(e >= 0 ? e : 0);
            (j & 1 ? wd[j / 2].y : wd[j / 2].x) = e >= 0 ? d : 0.f;
            (j & 1 ? wc[j / 2].y : wc[j / 2].x) = power(rev ? j : 31 - j);
        }
        const int J0 = rev ? R : 0, J1 = rev ? 3 : R;     // the 32-column blocks that the mask leaves
        for (int c = 0; !STATE && c < nch; ++c) {
            const int s = c & 1;
            if (!waitw(BAR(p_raw, s), (c >> 1) & 1)) break;
            tc_fence_after();
            const uint32_t tP = tmem + lane_base + kColP + s * 128;
#pragma unroll 1
            for (int J = 0; J < 4; ++J) {
                uint32_t o[16];
                if (J < J0 || J > J1) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = 0;
                } else {
                    float v[32];
                    tc_ld_32x32b_x32(tP + 32 * J, v);
                    wait_loaded(v);
                    if (J == R) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 p = __fmul2_rn(make_float2(v[2 * i], v[2 * i + 1]), wd[i]);
                            o[i] = pack_bf16x2(p.x, p.y);
                        }
                    } else {
                        const float rf = power(rev ? 32 * J - row : row - 32 * J - 31);
                        const float2 rf2 = make_float2(rf, rf);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 p = __fmul2_rn(make_float2(v[2 * i], v[2 * i + 1]), __fmul2_rn(wc[i], rf2));
                            o[i] = pack_bf16x2(p.x, p.y);
                        }
                    }
                }
                // (P's columns 16 J .. lie over scores of blocks <= J / 2, which this warp has read)
                tc_st_x16(tP + 16 * J, o);
            }
            tc_wait_st();
            tc_fence_before();
            bar_arrive_warp(BAR(p_ready, s));
        }
    } else if (group == 2) {
        // ------------------------------------------------ weighted values
        regs_dec<kRegsValues>();
        const uint32_t tW = s0 + L::kOffW;
        for (int c = 0; c < nch; ++c) {
            const int s = c % kStC, n = chunk_n(c);
            const uint32_t tC = sC + s * kBlk;
            const bool in = row < n;
            const float w = in ? power(rev ? row + 1 : n - 1 - row) * sw.write_scale : 0.f;
            const float2 w2 = make_float2(w, w), nw2 = make_float2(-w, -w);
            if (!waitw(BAR(fullC, s), (c / kStC) & 1)) break;
            if (packed && n < kCT) {
                // the rows behind the sequence are another's (or nobody's): they become zeros in b and c
                if (!waitw(BAR(fullB, c & 1), (c >> 1) & 1)) break;
                if (!in) {
#pragma unroll 1
                    for (int x = 0; x < 8; ++x) {
                        sts4(tC + sw128_offset(row, x), 0, 0, 0, 0);
                        for (int k = 0; k < L::NB; ++k)
                            sts4(sB + (c & 1) * L::kTile + k * kBlk + sw128_offset(row, x), 0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                bar_arrive_warp(BAR(tail, 0));
            }
            // both parts are formed while dS of chunk c - 1 still reads its own
            uint32_t hi[32], lo[32];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const uint4 raw = lds4(tC + sw128_offset(row, x));
                const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // the second part is what the first leaves of the exact product, with its sign turned
                    const float2 v = make_float2(bf16_lo(u[e]), bf16_hi(u[e]));
                    const float2 p = __fmul2_rn(v, w2);
                    const uint32_t q = pack_bf16x2(p.x, p.y);
                    const float2 d = __ffma2_rn(v, nw2, make_float2(bf16_lo(q), bf16_hi(q)));
                    hi[4 * x + e] = q;
                    lo[4 * x + e] = pack_bf16x2(d.x, d.y);
                }
            }
            if (c >= 1 && !waitw(BAR(w_empty, 0), (c - 1) & 1)) break;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const uint32_t at = sw128_offset(row, x);
                sts4(tW + at, hi[4 * x], hi[4 * x + 1], hi[4 * x + 2], hi[4 * x + 3]);
                sts4(tW + kBlk + at, lo[4 * x], lo[4 * x + 1], lo[4 * x + 2], lo[4 * x + 3]);
            }
            fence_proxy_async_smem();
            bar_arrive_warp(BAR(w_full, 0));
            if (STATE) bar_arrive_warp(BAR(emptyC, s));
        }
    } else {
        // ---------------------------------------------- state and outputs
        regs_inc<kRegsState>();
        const bool mine = row < KD;    // (ra = 64: the other rows hold what the unused rows of dS give)
        float2 S[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) S[j] = make_float2(0.f, 0.f);
        // the state that enters: S_init for a whole sweep and for the first part of a split one; a segment
        // takes what the parts before it leave, the first one the copy of S_init that the first part makes (S_fin
        // may lie over S_init, and the last segment may end before the first one begins)
        const size_t slots = args.nparts + 1;
        float *const parts = args.parts + ((bh * gridDim.x + blockIdx.x) * slots * KD + (row & (KD - 1))) * 64;
        if (sw.S_init && (STATE ? z == 0 : args.nseg == 1)) {
            // element j of the row: contiguous, or a row of the transposed state apart
            const int i = row & (KD - 1);
            const float *src = sw.init_t ? sw.S_init + (bh * n_all + c0) * KD + i : sw.S_init + (bh * KD + i) * n_all + c0;
            const size_t step = sw.init_t ? KD : 1;
            if (!sw.init_t && (reinterpret_cast<uintptr_t>(src) & 15) == 0) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float4 d = reinterpret_cast<const float4 *>(src)[j];
                    S[2 * j] = make_float2(d.x, d.y), S[2 * j + 1] = make_float2(d.z, d.w);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) S[j] = make_float2(src[2 * j * step], src[(2 * j + 1) * step]);
            }
        }
        if (STATE && z == 0 && mine) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                reinterpret_cast<float4 *>(parts + (size_t)args.nparts * KD * 64)[j] = make_float4(S[2 * j].x, S[2 * j].y, S[2 * j + 1].x, S[2 * j + 1].y);
        }
        if (!STATE && args.nseg > 1) {
            const int first = z ? 0 : args.nparts, end = z ? z * (args.seg_chunks / args.part_chunks) : first + 1;
            const float2 g2 = make_float2(sm->gpart, sm->gpart);
#pragma unroll 1
            for (int q = first; q < end; ++q) {
                const float4 *src = reinterpret_cast<const float4 *>(parts + (size_t)q * KD * 64);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float4 d = src[j];
                    S[2 * j] = __ffma2_rn(g2, S[2 * j], make_float2(d.x, d.y));
                    S[2 * j + 1] = __ffma2_rn(g2, S[2 * j + 1], make_float2(d.z, d.w));
                }
            }
        }
        auto publish = [&]() {
            const uint32_t tS = s0 + L::kOffS;
#pragma unroll
            for (int x = 0; x < 8; ++x)
                sts4(tS + sw128_offset(row, x), pack_bf16x2(S[4 * x].x, S[4 * x].y), pack_bf16x2(S[4 * x + 1].x, S[4 * x + 1].y),
                     pack_bf16x2(S[4 * x + 2].x, S[4 * x + 2].y), pack_bf16x2(S[4 * x + 3].x, S[4 * x + 3].y));
            fence_proxy_async_smem();
            bar_arrive_warp(BAR(s_full, 0));
        };
        const float s_in = sw.out_scale * sw.write_scale;
        const float2 si2 = make_float2(s_in, s_in);
        uint16_t *out = static_cast<uint16_t *>(sw.out);
        const int r0 = (warp & 3) * 32;    // this warp's rows of a tile
        bool ok = true;
        for (int c = 0; c <= nch; ++c) {
            float ye[64];
            if (!STATE && c >= 1) {
                // Ye of chunk c - 1 moves to registers, which frees its accumulator and the state's tile
                ok = waitw(BAR(ye_full, 0), (c - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                float(&y0)[32] = *reinterpret_cast<float(*)[32]>(ye), (&y1)[32] = *reinterpret_cast<float(*)[32]>(ye + 32);
                tc_ld_32x32b_x32(tmem + lane_base + kColYe, y0);
                tc_ld_32x32b_x32(tmem + lane_base + kColYe + 32, y1);
                wait_loaded(y0);
                wait_loaded(y1);
                tc_fence_before();
            }
            if (!STATE && c < nch) publish();
            if (!STATE && c >= 1) {
                // the outputs of chunk c - 1
                const int n = chunk_n(c - 1), t0 = chunk_t0(c - 1);
                const int e = rev ? n - 1 - row : row + 1;
                const float s_ex = sw.out_scale * power(e >= 0 ? e : 0);
                const float2 se2 = make_float2(s_ex, s_ex);
                // the rows leave through the chunk's own tile of c: Yi has read it, and so has the weighting
                // of its values (dS of this chunk was waited for)
                const uint32_t tY = sC + ((c - 1) % kStC) * kBlk;
                ok = waitw(BAR(yi_full, 0), (c - 1) & 1);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int x = 0; x < 64; x += 32) {
                    float yi[32];
                    tc_ld_32x32b_x32(tmem + lane_base + kColYi + x, yi);
                    wait_loaded(yi);
                    if (x == 32) {
                        tc_fence_before();
                        bar_arrive_warp(BAR(yi_empty, 0));
                    }
                    uint32_t o[16];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float2 y = __ffma2_rn(si2, make_float2(yi[j], yi[j + 1]),
                                                    __fmul2_rn(se2, make_float2(ye[x + j], ye[x + j + 1])));
                        o[j / 2] = pack_bf16x2(y.x, y.y);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        sts4(tY + sw128_offset(row, x / 8 + q), o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                }
                if (packed && n < kCT) {
                    // only the sequence's own rows, 8 lanes each
                    __syncwarp();
#pragma unroll 1
                    for (int r = r0 + (lane >> 3); r < min(n, r0 + 32); r += 4)
                        *reinterpret_cast<uint4 *>(out + ((size_t)(seq0 + t0 + r) * H + h) * n_all + c0 + (lane & 7) * 8) =
                            lds4(tY + sw128_offset(r, lane & 7));
                } else {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && r0 < n) {    // (rows behind the end of a sequence of its own are not written)
                        tma_store(&maps.out, tY + r0 * 128, c0, packed ? h : t0 + r0, packed ? seq0 + t0 + r0 : (int)bh);
                        tma_store_commit();
                    }
                }
            }
            if (c < nch) {
                const float gn = power(chunk_n(c));
                ok = waitw(BAR(ds_full, 0), c & 1);
                if (!ok) break;
                tc_fence_after();
                const float2 gn2 = make_float2(gn, gn), minus = make_float2(-1.f, -1.f);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float hi[32], lo[32];
                    tc_ld_32x32b_x32(tmem + lane_base + kColDS + 32 * x, hi);
                    tc_ld_32x32b_x32(tmem + lane_base + kColDS + 64 + 32 * x, lo);
                    wait_loaded(hi);
                    wait_loaded(lo);
                    if (x == 1) {
                        tc_fence_before();
                        bar_arrive_warp(BAR(ds_empty, 0));
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j)    // (the second part's sign is turned)
                        S[16 * x + j] = __ffma2_rn(gn2, S[16 * x + j],
                                                   __ffma2_rn(minus, make_float2(lo[2 * j], lo[2 * j + 1]),
                                                              make_float2(hi[2 * j], hi[2 * j + 1])));
                }
            }
            if (!STATE && c >= 1) {
                // the rows that left through chunk c - 1's tile have been read: the tile may be filled again
                if (lane == 0) tma_store_wait_read<0>();
                bar_arrive_warp(BAR(emptyC, (c - 1) % kStC));
            }
        }
        if (lane == 0) tma_store_wait_all<0>();
        __syncwarp();
        const bool last = cb + nch == all;
        if (ok && mine && (STATE || (sw.S_fin && last))) {
            float *dst = STATE ? parts + (size_t)z * KD * 64 : sw.S_fin + (bh * KD + row) * n_all + c0;
            if ((reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
#pragma unroll
                for (int j = 0; j < 32; j += 2)
                    *reinterpret_cast<float4 *>(dst + 2 * j) = make_float4(S[j].x, S[j].y, S[j + 1].x, S[j + 1].y);
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) dst[2 * j] = S[j].x, dst[2 * j + 1] = S[j].y;
            }
        }
    }
    // ------------------------------------------------------------ teardown
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && sm->abort_flag) atomicExch(args.d.status, kStatusTimeout);
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int KD, bool PACKED, bool REV, bool STATE>
cudaError_t launch(const DecayTcParams &p, cudaStream_t stream)
{
    static OncePerDevice once;
    const cudaError_t e = set_smem_once(decay_tc_kernel<KD, PACKED, REV, STATE>, smem_bytes<KD>(), once);
    if (e != cudaSuccess) return e;
    const dim3 grid(p.tiles[0] + p.tiles[1] + p.tiles[2], p.d.H, p.B * (STATE ? p.nparts : p.nseg));
    decay_tc_kernel<KD, PACKED, REV, STATE><<<grid, kThreads, smem_bytes<KD>(), stream>>>(p);
    return cudaGetLastError();
}

template <int KD, bool REV>
cudaError_t launch_dense(const DecayTcParams &p, cudaStream_t stream)
{
    if (p.nseg > 1)
        if (const cudaError_t e = launch<KD, false, REV, true>(p, stream)) return e;
    return launch<KD, false, REV, false>(p, stream);
}

template <int KD>
cudaError_t launch(const DecayTcParams &p, cudaStream_t stream)
{
    bool rev = false;
    for (int i = 0; i < 3; ++i) rev = rev || (p.tiles[i] && p.sw[i].rev);
    if (p.d.cu_seqlens) return launch<KD, true, false, false>(p, stream);
    return rev ? launch_dense<KD, true>(p, stream) : launch_dense<KD, false>(p, stream);
}

}  // namespace

cudaError_t launch_decay_tc(const DecayTcParams &p, int ra, cudaStream_t stream)
{
    return ra == 64 ? launch<64>(p, stream) : launch<128>(p, stream);
}

}  // namespace la
