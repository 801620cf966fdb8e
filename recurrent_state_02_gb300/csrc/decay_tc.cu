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
// and out = s_in Yi + s_out g^.. Ye leaves through a TMA store.
//
// The state is FP32 in the registers of four warps: after each chunk S <- g^n S + dS
// (both halves), so that its rounding is that of one FP32 sum per chunk.  Two
// BF16 parts of the weighted values keep the state to 2^-16 per term, where one
// part would leave 2^-8; the outputs, which are BF16, take P and S rounded once.
//
// No power of g is ever divided by: a block of 32 x 32 scores below the diagonal carries
// g^{p_i - p_j} as the product of a row's power and a column's power, both with
// exponents >= 0; a diagonal block looks its powers up.  So every g in 0 .. 1 (0 too)
// takes the same path, and what underflows is negligible next to the diagonal.
//
// One CTA owns one (b, h, 64 columns of c) and walks its chunks.  18 warps: TMA
// producer, MMA issuer, and four groups of four (each warp reaches the TMEM lanes of its
// quadrant, warp % 4): scores, weighted values, state, outputs.
#include "decay.h"
#include "tc_common.cuh"

namespace la {
namespace {

constexpr int kCT = 128;                       // tokens per chunk
constexpr int kThreads = 18 * 32;
constexpr int kWarpTma = 0, kWarpMma = 1, kGroupP = 2, kGroupC = 6, kGroupS = 10, kGroupY = 14;   // first warps
constexpr uint32_t kBlk = kCT * 128;           // 16 KB: 128 rows x 64 BF16 columns, 128-byte swizzle
constexpr int kNST = 2;

// TMEM columns
constexpr uint32_t kColP = 0, kColYi = 256, kColYe = 320, kColDS = 384;

template <int KD>
struct Lay {
    static constexpr int NB = KD / 64;                       // 64-column blocks of a and b
    static constexpr uint32_t kA = 0, kB = NB * kBlk, kC = 2 * NB * kBlk;
    static constexpr uint32_t kStage = (2 * NB + 1) * kBlk;
    static constexpr uint32_t kOffW = kNST * kStage;         // weighted values: Ch, Cl
    static constexpr uint32_t kOffS = kOffW + 2 * kBlk;      // the state as BF16 [KD x 64]
    static constexpr uint32_t kOffY = kOffS + KD * 128;      // output tile
    static constexpr uint32_t kOffSmall = kOffY + kBlk;
};

struct alignas(16) SmallD {
    uint64_t fullA[kNST], fullB[kNST], fullC[kNST], emptyA[kNST], emptyB[kNST], emptyC[kNST];
    uint64_t p_raw[2], p_ready[2], w_full, w_empty, ds_full, ds_empty, s_full, s_empty, y_full, y_empty, t_free, t_full, done;
    uint32_t tmem_base;
    int abort_flag;
    int seq;
    alignas(16) float pw[kCT + 4];     // g^0 .. g^128
    alignas(16) float col[32];         // a block's column powers
};

template <int KD>
constexpr uint32_t smem_bytes() { return Lay<KD>::kOffSmall + sizeof(SmallD) + 1024; }
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory budget");

// D[tmem] (+)= A[tmem] * B[smem]
template <bool ACC>
__device__ __forceinline__ void tc_mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "n"(ACC ? 1 : 0)
        : "memory");
}

// 32 lanes x 32 bits, 8 consecutive columns.
__device__ __forceinline__ void tc_ld_x8(uint32_t taddr, float (&v)[8])
{
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tc_st_x16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
          "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
          "r"(r[15])
        : "memory");
}

template <int KD>
__global__ void __launch_bounds__(kThreads, 1)
decay_tc_kernel(const __grid_constant__ DecayTcParams args)
{
    using L = Lay<KD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    SmallD *sm = reinterpret_cast<SmallD *>(base + L::kOffSmall);
    Ctx cx{&sm->abort_flag, args.wait_limit_ns, args.d.status};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    int tile = blockIdx.x, which = 0;
    while (tile >= args.tiles[which]) tile -= args.tiles[which++];
    const DecaySweep &sw = args.sw[which];
    const TcSweepMaps &maps = args.maps[which];
    const int h = blockIdx.y, H = args.d.H, n_all = sw.n, c0 = tile * 64;
    const bool rev = sw.rev, packed = args.d.cu_seqlens != nullptr;

    // this CTA's sequence
    int b = blockIdx.z, T = args.d.T, seq0 = 0;
    if (packed) {
        seq0 = args.d.cu_seqlens[b];
        const int seq1 = args.d.cu_seqlens[b + 1];
        // (bad bounds are recorded by the token kernel's launch, which looks at every sequence)
        if (seq0 < 0 || seq1 < seq0 || seq1 > args.d.T) return;
        T = seq1 - seq0;
        if (T < args.d.len_min || T > args.d.len_max) return;
    }
    const size_t bh = (size_t)b * H + h;
    const int nch = (T + kCT - 1) / kCT;
    // chunk of the sweep's step c, its first token and its tokens
    auto chunk_t0 = [&](int c) { return (rev ? nch - 1 - c : c) * kCT; };
    auto chunk_n = [&](int c) { return min(kCT, T - chunk_t0(c)); };

    // ------------------------------------------------------------ set-up
    if (tid == 0) {
        for (int s = 0; s < kNST; ++s) {
            for (uint64_t *bar : {&sm->fullA[s], &sm->fullB[s], &sm->fullC[s], &sm->emptyA[s], &sm->emptyB[s], &sm->emptyC[s]})
                mbar_init(bar, 1);
            mbar_init(&sm->p_raw[s], 1);
            mbar_init(&sm->p_ready[s], 4);
        }
        mbar_init(&sm->w_full, 4);
        mbar_init(&sm->w_empty, 1);
        mbar_init(&sm->ds_full, 1);
        mbar_init(&sm->ds_empty, 4);
        mbar_init(&sm->s_full, 4);
        mbar_init(&sm->s_empty, 1);
        mbar_init(&sm->y_full, 1);
        mbar_init(&sm->y_empty, 4);
        mbar_init(&sm->t_free, 1);
        mbar_init(&sm->t_full, 4);
        mbar_init(&sm->done, 1);
        sm->abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&maps.a);
        tma_prefetch_desc(&maps.b);
        tma_prefetch_desc(&maps.c);
        tma_prefetch_desc(&maps.out);
    }
    if (warp == kWarpMma) {
        tmem_alloc(&sm->tmem_base, 512);
        tmem_relinquish();
    }
    if (tid >= 64 && tid - 64 <= kCT) {
        // powers of g from its repeated squares in 64 bits: each entry is rounded once
        const int e = tid - 64;
        double p = 1.0, q = (double)args.d.decay[h];
        for (int bit = 0; bit < 8; ++bit) {
            if (e >> bit & 1) p *= q;
            q *= q;
        }
        sm->pw[e] = (float)p;
        if (e < 32) sm->col[rev ? e : 31 - e] = (float)p;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm->tmem_base;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int row = (warp & 3) * 32 + lane;     // the TMEM lane, and tile row, of this thread

    if (warp == kWarpTma) {
        // ------------------------------------------------------- producer
        int issued = 0;
        if (lane == 0) {
            for (int c = 0; c < nch; ++c) {
                const int s = c & 1, t0 = chunk_t0(c);
                const uint32_t ph = ((c >> 1) - 1) & 1;
                const int cy = packed ? h : t0, cz = packed ? seq0 + t0 : (int)bh;
                uint8_t *st = base + s * L::kStage;
                if (c >= kNST && !wait(cx, &sm->emptyB[s], ph)) break;
                mbar_arrive_expect_tx(&sm->fullB[s], L::NB * kBlk);
#pragma unroll
                for (int k = 0; k < L::NB; ++k) tma_load_3d(st + L::kB + k * kBlk, &maps.b, &sm->fullB[s], 64 * k, cy, cz);
                issued = 3 * c + 1;
                if (c >= kNST && !wait(cx, &sm->emptyC[s], ph)) break;
                mbar_arrive_expect_tx(&sm->fullC[s], kBlk);
                tma_load_3d(st + L::kC, &maps.c, &sm->fullC[s], c0, cy, cz);
                issued = 3 * c + 2;
                if (c >= kNST && !wait(cx, &sm->emptyA[s], ph)) break;
                mbar_arrive_expect_tx(&sm->fullA[s], L::NB * kBlk);
#pragma unroll
                for (int k = 0; k < L::NB; ++k) tma_load_3d(st + L::kA + k * kBlk, &maps.a, &sm->fullA[s], 64 * k, cy, cz);
                issued = 3 * c + 3;
            }
            if (aborted(cx)) {
                // every issued load lands before the CTA may exit
                for (int i = issued > 6 ? issued - 6 : 0; i < issued; ++i) {
                    const int c = i / 3, k = i % 3;
                    uint64_t *bar = k == 0 ? &sm->fullB[c & 1] : k == 1 ? &sm->fullC[c & 1] : &sm->fullA[c & 1];
                    mbar_wait(bar, (c >> 1) & 1, cx.limit);
                }
            }
        }
        __syncwarp();
    } else if (warp == kWarpMma) {
        // ------------------------------------------------------------ MMA
        if (lane == 0) {
            constexpr uint32_t idP = idesc_bf16_f32(128, 128, false, false);
            constexpr uint32_t idY = idesc_bf16_f32(128, 64, false, true);
            constexpr uint32_t idDS = idesc_bf16_f32(128, 128, true, true);
            constexpr uint32_t kHi = desc_hi(1024, 2);
            // scores of chunk c; their buffer held P of chunk c - 2, whose product is done
            auto issue_p = [&](int c) -> bool {
                const int s = c & 1;
                if (!wait(cx, &sm->fullA[s], (c >> 1) & 1) || !wait(cx, &sm->fullB[s], (c >> 1) & 1)) return false;
                if (c >= 2 && !wait(cx, &sm->y_full, (c - 2) & 1)) return false;
                tc_fence_after();
                const uint32_t st = smem_u32(base + s * L::kStage);
                const uint32_t alo = desc_lo(st + L::kA, 16), blo = desc_lo(st + L::kB, 16), d = tmem + kColP + s * 128;
#pragma unroll
                for (int k = 0; k < KD / 16; ++k) {
                    const uint32_t o = ((k >> 2) * kBlk + (k & 3) * 32) >> 4;
                    if (k == 0) tc_mma_bf16_w<false>(d, alo, kHi, blo, kHi, idP);
                    else tc_mma_bf16_w<true>(d, alo + o, kHi, blo + o, kHi, idP);
                }
                tc_commit(&sm->p_raw[s]);
                return true;
            };
            bool ok = nch == 0 || issue_p(0);
            for (int c = 0; c < nch && ok; ++c) {
                const int s = c & 1;
                const uint32_t st = smem_u32(base + s * L::kStage);
                // dS = B^T [Ch | Cl]
                if (!wait(cx, &sm->w_full, c & 1)) break;
                if (c >= 1 && !wait(cx, &sm->ds_empty, (c - 1) & 1)) break;
                tc_fence_after();
                {
                    // (ra = 64: rows 64 .. 127 of the product come from the tile behind b and are not used)
                    const uint32_t alo = desc_lo(st + L::kB, kBlk), blo = desc_lo(smem_u32(base + L::kOffW), kBlk);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t o = k * (2048 >> 4);
                        if (k == 0) tc_mma_bf16_w<false>(tmem + kColDS, alo, kHi, blo, kHi, idDS);
                        else tc_mma_bf16_w<true>(tmem + kColDS, alo + o, kHi, blo + o, kHi, idDS);
                    }
                }
                tc_commit(&sm->ds_full);
                tc_commit(&sm->w_empty);
                tc_commit(&sm->emptyB[s]);   // (the scores read b before)
                if (c + 1 < nch && !issue_p(c + 1)) break;
                // Ye = A S
                if (!wait(cx, &sm->s_full, c & 1)) break;
                if (c >= 1 && !wait(cx, &sm->y_empty, (c - 1) & 1)) break;
                tc_fence_after();
                {
                    const uint32_t alo = desc_lo(st + L::kA, 16), blo = desc_lo(smem_u32(base + L::kOffS), kBlk);
#pragma unroll
                    for (int k = 0; k < KD / 16; ++k) {
                        const uint32_t o = ((k >> 2) * kBlk + (k & 3) * 32) >> 4;
                        if (k == 0) tc_mma_bf16_w<false>(tmem + kColYe, alo, kHi, blo, kHi, idY);
                        else tc_mma_bf16_w<true>(tmem + kColYe, alo + o, kHi, blo + k * (2048 >> 4), kHi, idY);
                    }
                }
                tc_commit(&sm->s_empty);
                tc_commit(&sm->emptyA[s]);
                // Yi = P C
                if (!wait(cx, &sm->p_ready[s], (c >> 1) & 1)) break;
                tc_fence_after();
                {
                    const uint32_t blo = desc_lo(st + L::kC, kBlk), a = tmem + kColP + s * 128;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (k == 0) tc_mma_bf16_ts<false>(tmem + kColYi, a, blo, kHi, idY);
                        else tc_mma_bf16_ts<true>(tmem + kColYi, a + 8 * k, blo + k * (2048 >> 4), kHi, idY);
                    }
                }
                tc_commit(&sm->y_full);
                tc_commit(&sm->emptyC[s]);
            }
            // every MMA issued above completes before TMEM is released
            tc_commit(&sm->done);
            mbar_wait(&sm->done, 0, cx.limit);
        }
        __syncwarp();
    } else if (warp < kGroupC) {
        // --------------------------------------------------------- scores
        const int R = warp & 3;
        const float *pw = sm->pw;
        for (int c = 0; c < nch; ++c) {
            const int s = c & 1;
            if (!warp_wait(cx, &sm->p_raw[s], (c >> 1) & 1)) break;
            tc_fence_after();
            const uint32_t tP = tmem + lane_base + kColP + s * 128;
#pragma unroll 1
            for (int J = 0; J < 4; ++J) {
                uint32_t o[16];
                if (rev ? J < R : J > R) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = 0;
                } else {
                    float v[32];
                    tc_ld_32x32b_x32(tP + 32 * J, v);
                    tc_wait_ld();
                    if (J == R) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const int e = rev ? j - lane : lane - j;
                            v[j] = e >= 0 ? v[j] * pw[e >= 0 ? e : 0] : 0.f;
                        }
                    } else {
                        const float rf = pw[rev ? 32 * J - row : row - 32 * J - 31];
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 cf = *reinterpret_cast<const float4 *>(sm->col + j);
                            v[j] *= rf * cf.x, v[j + 1] *= rf * cf.y, v[j + 2] *= rf * cf.z, v[j + 3] *= rf * cf.w;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
                }
                // (P's columns 16 J .. overwrite scores of blocks <= J, which this warp has read)
                tc_st_x16(tP + 16 * J, o);
            }
            tc_wait_st();
            tc_fence_before();
            warp_arrive(&sm->p_ready[s]);
        }
    } else if (warp < kGroupS) {
        // ------------------------------------------------ weighted values
        for (int c = 0; c < nch; ++c) {
            const int s = c & 1, n = chunk_n(c);
            if (!warp_wait(cx, &sm->fullC[s], (c >> 1) & 1)) break;
            uint8_t *tC = base + s * L::kStage + L::kC;
            const bool in = row < n;
            const float w = in ? sm->pw[rev ? row + 1 : n - 1 - row] * sw.write_scale : 0.f;
            uint4 raw[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) raw[x] = *reinterpret_cast<const uint4 *>(tC + sw128_offset(row, x));
            if (packed && n < kCT) {
                // the rows behind the sequence are another's (or nobody's): they become zeros in b and c
                if (!warp_wait(cx, &sm->fullB[s], (c >> 1) & 1)) break;
                if (!in) {
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        raw[x] = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(tC + sw128_offset(row, x)) = raw[x];
#pragma unroll
                        for (int k = 0; k < L::NB; ++k)
                            *reinterpret_cast<uint4 *>(base + s * L::kStage + L::kB + k * kBlk + sw128_offset(row, x)) = raw[x];
                    }
                }
            }
            if (c >= 1 && !warp_wait(cx, &sm->w_empty, (c - 1) & 1)) break;
            uint8_t *tW = base + L::kOffW;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const uint32_t u[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float f0 = bf16_lo(u[e]) * w, f1 = bf16_hi(u[e]) * w;
                    hi[e] = pack_bf16x2(f0, f1);
                    lo[e] = pack_bf16x2(f0 - bf16_lo(hi[e]), f1 - bf16_hi(hi[e]));
                }
                *reinterpret_cast<uint4 *>(tW + sw128_offset(row, x)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(tW + kBlk + sw128_offset(row, x)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            fence_proxy_async_smem();
            warp_arrive(&sm->w_full);
        }
    } else if (warp < kGroupY) {
        // ---------------------------------------------------------- state
        const bool mine = row < KD;    // (ra = 64: two of the four warps)
        float S[64];
#pragma unroll
        for (int j = 0; j < 64; ++j) S[j] = 0.f;
        if (mine && sw.S_init) {
            if (sw.init_t) {
                const float *src = sw.S_init + (bh * n_all + c0) * KD + row;
#pragma unroll
                for (int j = 0; j < 64; ++j) S[j] = src[(size_t)j * KD];
            } else {
                const float *src = sw.S_init + (bh * KD + row) * n_all + c0;
                if ((reinterpret_cast<uintptr_t>(src) & 15) == 0) {
#pragma unroll
                    for (int j = 0; j < 64; j += 4) {
                        const float4 q = *reinterpret_cast<const float4 *>(src + j);
                        S[j] = q.x, S[j + 1] = q.y, S[j + 2] = q.z, S[j + 3] = q.w;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 64; ++j) S[j] = src[j];
                }
            }
        }
        auto publish = [&]() {
            if (mine) {
                uint8_t *tS = base + L::kOffS;
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    *reinterpret_cast<uint4 *>(tS + sw128_offset(row, x)) =
                        make_uint4(pack_bf16x2(S[8 * x], S[8 * x + 1]), pack_bf16x2(S[8 * x + 2], S[8 * x + 3]),
                                   pack_bf16x2(S[8 * x + 4], S[8 * x + 5]), pack_bf16x2(S[8 * x + 6], S[8 * x + 7]));
            }
            fence_proxy_async_smem();
            warp_arrive(&sm->s_full);
        };
        if (nch > 0) publish();
        bool ok = true;
        for (int c = 0; c < nch; ++c) {
            const float gn = sm->pw[chunk_n(c)];
            ok = warp_wait(cx, &sm->ds_full, c & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < 64; x += 8) {
                float hi[8], lo[8];
                tc_ld_x8(tmem + lane_base + kColDS + x, hi);
                tc_ld_x8(tmem + lane_base + kColDS + 64 + x, lo);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j) S[x + j] = fmaf(gn, S[x + j], hi[j] + lo[j]);
            }
            tc_fence_before();
            warp_arrive(&sm->ds_empty);
            if (c + 1 < nch) {
                ok = warp_wait(cx, &sm->s_empty, c & 1);
                if (!ok) break;
                publish();
            }
        }
        if (ok && mine && sw.S_fin) {
            float *dst = sw.S_fin + (bh * KD + row) * n_all + c0;
            if ((reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
#pragma unroll
                for (int j = 0; j < 64; j += 4)
                    *reinterpret_cast<float4 *>(dst + j) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < 64; ++j) dst[j] = S[j];
            }
        }
    } else {
        // -------------------------------------------------------- outputs
        const float s_in = sw.out_scale * sw.write_scale;
        uint8_t *tY = base + L::kOffY;
        for (int c = 0; c < nch; ++c) {
            const int n = chunk_n(c), t0 = chunk_t0(c);
            const int e = rev ? n - 1 - row : row + 1;
            const float s_ex = sw.out_scale * sm->pw[e >= 0 ? e : 0];
            if (!warp_wait(cx, &sm->y_full, c & 1)) break;
            tc_fence_after();
            uint32_t o[32];
#pragma unroll
            for (int x = 0; x < 64; x += 16) {
                float yi[16], ye[16];
                tc_ld_32x32b_x16(tmem + lane_base + kColYi + x, yi);
                tc_ld_32x32b_x16(tmem + lane_base + kColYe + x, ye);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; j += 2)
                    o[(x + j) / 2] = pack_bf16x2(fmaf(s_in, yi[j], s_ex * ye[j]), fmaf(s_in, yi[j + 1], s_ex * ye[j + 1]));
            }
            tc_fence_before();
            warp_arrive(&sm->y_empty);
            // the tile is free once its last store has been read out of shared memory
            if (warp == kGroupY) {
                if (lane == 0) {
                    tma_store_wait_read<0>();
                    mbar_arrive(&sm->t_free);
                }
                __syncwarp();
            }
            if (!warp_wait(cx, &sm->t_free, c & 1)) break;
#pragma unroll
            for (int x = 0; x < 8; ++x)
                *reinterpret_cast<uint4 *>(tY + sw128_offset(row, x)) = make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
            if (packed && n < kCT) {
                // only the sequence's own rows: each warp its 32, 8 lanes per row
                __syncwarp();
                uint16_t *y = static_cast<uint16_t *>(sw.out);
                const int r0 = (warp & 3) * 32;
                for (int r = r0 + (lane >> 3); r < min(n, r0 + 32); r += 4)
                    *reinterpret_cast<uint4 *>(y + ((size_t)(seq0 + t0 + r) * H + h) * n_all + c0 + (lane & 7) * 8) =
                        *reinterpret_cast<const uint4 *>(tY + sw128_offset(r, lane & 7));
            } else {
                fence_proxy_async_smem();
                warp_arrive(&sm->t_full);
                if (warp == kGroupY) {
                    if (!warp_wait(cx, &sm->t_full, c & 1)) break;
                    if (lane == 0) {
                        tma_store_3d(&maps.out, tY, c0, packed ? h : t0, packed ? seq0 + t0 : (int)bh);
                        tma_store_commit();
                    }
                    __syncwarp();
                }
            }
        }
        if (warp == kGroupY && lane == 0) tma_store_wait_all<0>();
        __syncwarp();
    }
    // ------------------------------------------------------------ teardown
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

template <int KD>
cudaError_t launch(const DecayTcParams &p, cudaStream_t stream)
{
    static OncePerDevice once;
    const cudaError_t e = set_smem_once(decay_tc_kernel<KD>, smem_bytes<KD>(), once);
    if (e != cudaSuccess) return e;
    const dim3 grid(p.tiles[0] + p.tiles[1] + p.tiles[2], p.d.H, p.B);
    decay_tc_kernel<KD><<<grid, kThreads, smem_bytes<KD>(), stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decay_tc(const DecayTcParams &p, int ra, cudaStream_t stream)
{
    return ra == 64 ? launch<64>(p, stream) : launch<128>(p, stream);
}

}  // namespace la
