// decay.cu -- linear attention with a constant decay per head on CUDA cores: the
// token recurrence (any sizes, FP32 arithmetic) and the single-token decode step.
//
//     S_t = g S_{t-1} + k_t v_t^T,   y_t = scale q_t^T S_t
//
// There is no feature map and no normaliser; g is a constant of the head.

#include "decay.h"
#include "sm103_ptx.cuh"

#include <cuda_bf16.h>

namespace la {
namespace {

template <bool BF16>
__device__ __forceinline__ float load_elem(const void *p, size_t i)
{
    if (BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
    return reinterpret_cast<const float *>(p)[i];
}

template <bool BF16>
__device__ __forceinline__ void store_elem(void *p, size_t i, float x)
{
    if (BF16) reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
    else reinterpret_cast<float *>(p)[i] = x;
}

// ------------------------------------------------------- token recurrence
// One CTA of 4 warps per (b, h, 64 columns), the state in registers: lane
// (g, jj), g = lane / 4, holds rows {4 (8 m + g) + e : m < RP/32, e < 4} of the
// four columns 4 jj .. 4 jj + 3 of its warp's 16.  A row's two operands come from
// shared memory as 16-byte words that serve four columns (the 8 groups of a warp
// read 128 different bytes), so a token costs a warp RP/16 shared loads
// for 3 RP/32 * 16 / 2 packed FP32 instructions: the FMA pipe is the limit, not
// shared memory.  The sums over rows are reduced two tokens at a time: 8 partial
// sums per lane (2 tokens x 4 columns) over the 8 row groups, by a
// reduce-scatter of 4 + 2 + 1 shuffles, which leaves each lane one total.
// Tokens are staged in blocks of TB; the next block's values are fetched
// into registers while this one is computed.
constexpr int kRecCols = 64, kRecThreads = 128;

template <int RP>
struct RecCfg {
    static constexpr int M = RP / 32;                 // float4 row blocks per lane
    static constexpr int TB = RP >= 256 ? 8 : 16;     // tokens per staged block
    static constexpr int RS = RP + 4;                 // row stride of the staged a, b (floats)
    static constexpr int NA = TB * RP / kRecThreads;  // staged a (or b) values per thread
    static constexpr int NC = TB * kRecCols / kRecThreads;
};

struct RecArgs {
    DecaySweep sw[3];
    DecayArgs d;
    int tiles[3];   // column tiles of each sweep
};

__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }

template <bool BF16, int RP>
__global__ void __launch_bounds__(kRecThreads)
decay_rec_kernel(const __grid_constant__ RecArgs args)
{
    using C = RecCfg<RP>;
    constexpr int M = C::M, TB = C::TB, RS = C::RS;
    __shared__ float4 as4[TB * RS / 4], bs4[TB * RS / 4], cs4[TB * kRecCols / 4];
    __shared__ float ys[TB][kRecCols];
    float *as = reinterpret_cast<float *>(as4), *bs = reinterpret_cast<float *>(bs4),
          *cs = reinterpret_cast<float *>(cs4);
    int tile = blockIdx.x, which = 0;
    while (tile >= args.tiles[which]) tile -= args.tiles[which++];
    const DecaySweep &sw = args.sw[which];
    const DecayArgs &d = args.d;
    const int h = blockIdx.y, b = blockIdx.z, H = d.H, ra = sw.ra, n = sw.n;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, jj = lane & 3;
    const bool packed = d.cu_seqlens != nullptr;
    int T = d.T, seq0 = 0;
    if (packed) {
        seq0 = d.cu_seqlens[b];
        const int seq1 = d.cu_seqlens[b + 1];
        if (seq0 < 0 || seq1 < seq0 || seq1 > d.T) {
            if (tid == 0) atomicExch(d.status, kStatusShape);
            return;
        }
        T = seq1 - seq0;
        if (T < d.len_min || T > d.len_max) return;
    }
    const size_t bh = (size_t)b * H + h;
    // row (of ra or n elements) of the sweep's t-th token
    auto row = [&](int t) -> size_t {
        const int at = sw.rev ? T - 1 - t : t;
        return packed ? (size_t)(seq0 + at) * H + h : bh * T + at;
    };
    const float g = d.decay[h];
    const int c0 = tile * kRecCols, wc = warp * 16 + jj * 4;   // first column of the CTA; of the lane, inside it
    const bool active = c0 + warp * 16 < n;                    // (warp-uniform)

    // state rows 4 (8 m + g8) + e, columns c0 + wc + (0 .. 3) as two packed pairs
    float2 s[M][4][2];
    const bool vec = !sw.init_t && (n & 3) == 0 && (reinterpret_cast<uintptr_t>(sw.S_init) & 15) == 0;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 4 * (8 * m + g8) + e, j = c0 + wc;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (sw.S_init && i < ra && j < n) {
                const float *src = sw.S_init + bh * ra * n;
                if (vec) {
                    const float4 q4 = *reinterpret_cast<const float4 *>(src + (size_t)i * n + j);
                    v[0] = q4.x, v[1] = q4.y, v[2] = q4.z, v[3] = q4.w;
                } else {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (j + x < n) v[x] = sw.init_t ? src[(size_t)(j + x) * ra + i] : src[(size_t)i * n + j + x];
                }
            }
            s[m][e][0] = make_float2(v[0], v[1]);
            s[m][e][1] = make_float2(v[2], v[3]);
        }

    float pa[C::NA], pb[C::NA], pc[C::NC];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < C::NA; ++i) {
            const int x = i * kRecThreads + tid, t = t0 + x / RP, e = x % RP;
            const bool ok = t < T && e < ra;
            const size_t at = ok ? row(t) * ra + e : 0;
            pa[i] = ok ? load_elem<BF16>(sw.a, at) : 0.f;
            pb[i] = ok ? load_elem<BF16>(sw.b, at) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < C::NC; ++i) {
            const int x = i * kRecThreads + tid, t = t0 + x / kRecCols, e = c0 + x % kRecCols;
            const bool ok = t < T && e < n;
            pc[i] = ok ? load_elem<BF16>(sw.c, row(t) * n + e) * sw.write_scale : 0.f;
        }
    };
    if (T > 0) fetch(0);
    for (int t0 = 0; t0 < T; t0 += TB) {
        const int nt = min(TB, T - t0);
#pragma unroll
        for (int i = 0; i < C::NA; ++i) {
            const int x = i * kRecThreads + tid;
            as[(x / RP) * RS + x % RP] = pa[i];
            bs[(x / RP) * RS + x % RP] = pb[i];
        }
#pragma unroll
        for (int i = 0; i < C::NC; ++i) cs[i * kRecThreads + tid] = pc[i];
        __syncthreads();
        if (t0 + TB < T) fetch(t0 + TB);
        if (active) {
            for (int t = 0; t < nt; t += 2) {
                // (the second token of an odd last pair: zeros are staged, and a factor 1 keeps the state)
                const float2 f0 = splat((t0 + t == 0 && sw.late) ? 1.f : g), f1 = splat(t + 1 < nt ? g : 1.f);
                float2 y[2][2] = {};
                const float4 cv0 = *reinterpret_cast<const float4 *>(cs + t * kRecCols + wc);
                const float4 cv1 = *reinterpret_cast<const float4 *>(cs + (t + 1) * kRecCols + wc);
                const float2 c00 = make_float2(cv0.x, cv0.y), c01 = make_float2(cv0.z, cv0.w);
                const float2 c10 = make_float2(cv1.x, cv1.y), c11 = make_float2(cv1.z, cv1.w);
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const int o = 4 * (8 * m + g8);
                    const float4 a0 = *reinterpret_cast<const float4 *>(as + t * RS + o);
                    const float4 b0 = *reinterpret_cast<const float4 *>(bs + t * RS + o);
                    const float4 a1 = *reinterpret_cast<const float4 *>(as + (t + 1) * RS + o);
                    const float4 b1 = *reinterpret_cast<const float4 *>(bs + (t + 1) * RS + o);
                    const float aa0[4] = {a0.x, a0.y, a0.z, a0.w}, bb0[4] = {b0.x, b0.y, b0.z, b0.w};
                    const float aa1[4] = {a1.x, a1.y, a1.z, a1.w}, bb1[4] = {b1.x, b1.y, b1.z, b1.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float2 u = __ffma2_rn(f0, s[m][e][0], __fmul2_rn(splat(bb0[e]), c00));
                        float2 v = __ffma2_rn(f0, s[m][e][1], __fmul2_rn(splat(bb0[e]), c01));
                        y[0][0] = __ffma2_rn(splat(aa0[e]), u, y[0][0]);
                        y[0][1] = __ffma2_rn(splat(aa0[e]), v, y[0][1]);
                        u = __ffma2_rn(f1, u, __fmul2_rn(splat(bb1[e]), c10));
                        v = __ffma2_rn(f1, v, __fmul2_rn(splat(bb1[e]), c11));
                        y[1][0] = __ffma2_rn(splat(aa1[e]), u, y[1][0]);
                        y[1][1] = __ffma2_rn(splat(aa1[e]), v, y[1][1]);
                        s[m][e][0] = u;
                        s[m][e][1] = v;
                    }
                }
                // reduce-scatter over the row groups (lane bits 4, 3, 2): token, column pair, column
                const bool hi4 = lane & 16, hi3 = lane & 8, hi2 = lane & 4;
                float k0[4] = {hi4 ? y[1][0].x : y[0][0].x, hi4 ? y[1][0].y : y[0][0].y,
                               hi4 ? y[1][1].x : y[0][1].x, hi4 ? y[1][1].y : y[0][1].y};
                const float o0[4] = {hi4 ? y[0][0].x : y[1][0].x, hi4 ? y[0][0].y : y[1][0].y,
                                     hi4 ? y[0][1].x : y[1][1].x, hi4 ? y[0][1].y : y[1][1].y};
#pragma unroll
                for (int x = 0; x < 4; ++x) k0[x] += __shfl_xor_sync(0xffffffffu, o0[x], 16);
                float k1[2] = {hi3 ? k0[2] : k0[0], hi3 ? k0[3] : k0[1]};
                const float o1[2] = {hi3 ? k0[0] : k0[2], hi3 ? k0[1] : k0[3]};
#pragma unroll
                for (int x = 0; x < 2; ++x) k1[x] += __shfl_xor_sync(0xffffffffu, o1[x], 8);
                const float total = (hi2 ? k1[1] : k1[0]) + __shfl_xor_sync(0xffffffffu, hi2 ? k1[0] : k1[1], 4);
                ys[t + (hi4 ? 1 : 0)][wc + (hi3 ? 2 : 0) + (hi2 ? 1 : 0)] = total;
            }
        }
        __syncthreads();
        for (int x = tid; x < nt * kRecCols; x += kRecThreads) {
            const int t = x / kRecCols, e = x % kRecCols;
            if (c0 + e < n) store_elem<BF16>(sw.out, row(t0 + t) * n + c0 + e, ys[t][e] * sw.out_scale);
        }
        // (the next iteration's first barrier orders these reads of ys before its next writes, and
        // this iteration's last one its reads of the staged tokens before they are overwritten)
    }
    if (!sw.S_fin) return;
    const float2 f = splat(sw.late && T > 0 ? g : 1.f);
    const bool vec_out = (n & 3) == 0 && (reinterpret_cast<uintptr_t>(sw.S_fin) & 15) == 0;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 4 * (8 * m + g8) + e, j = c0 + wc;
            if (i >= ra || j >= n) continue;
            const float2 u = __fmul2_rn(s[m][e][0], f), v = __fmul2_rn(s[m][e][1], f);
            float *dst = sw.S_fin + bh * ra * n + (size_t)i * n + j;
            if (vec_out) {
                *reinterpret_cast<float4 *>(dst) = make_float4(u.x, u.y, v.x, v.y);
            } else {
                const float x[4] = {u.x, u.y, v.x, v.y};
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    if (j + w < n) dst[w] = x[w];
            }
        }
}

template <bool BF16>
cudaError_t launch_rec(const RecArgs &r, int rp, dim3 grid, cudaStream_t stream)
{
    if (rp <= 32) decay_rec_kernel<BF16, 32><<<grid, kRecThreads, 0, stream>>>(r);
    else if (rp <= 64) decay_rec_kernel<BF16, 64><<<grid, kRecThreads, 0, stream>>>(r);
    else if (rp <= 128) decay_rec_kernel<BF16, 128><<<grid, kRecThreads, 0, stream>>>(r);
    else decay_rec_kernel<BF16, 256><<<grid, kRecThreads, 0, stream>>>(r);
    return cudaGetLastError();
}

// ------------------------------------------------------------ decode step
// Reads and rewrites r dv FP32 state words per head, two FMAs each: bound by HBM.
// CTA (b, h) of 8 warps; a warp takes RW rows, its lanes 4 columns each, and
// issues every state load before any arithmetic.
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

template <bool BF16, int RW>
__global__ void __launch_bounds__(256)
decay_decode_kernel(const void *__restrict__ q, const void *__restrict__ k, const void *__restrict__ v,
                    const float *__restrict__ decay, float *__restrict__ S, int H, int r, int dv, float scale,
                    void *__restrict__ y)
{
    __shared__ float qs[8 * RW], ks[8 * RW];
    __shared__ float4 part[8][32];
    const size_t bh = blockIdx.x;
    const int c0 = blockIdx.y * 128;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int j = c0 + 4 * lane;
    const bool col = j < dv;
    float4 *Sr = reinterpret_cast<float4 *>(S + (bh * r + (size_t)warp * RW) * dv + (col ? j : 0));
    const int dv4 = dv >> 2;
    float4 s[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (col && warp * RW + i < r) s[i] = ld_stream(Sr + (size_t)i * dv4);
    }
    for (int i = tid; i < 8 * RW; i += 256) {
        qs[i] = i < r ? load_elem<BF16>(q, bh * r + i) : 0.f;
        ks[i] = i < r ? load_elem<BF16>(k, bh * r + i) : 0.f;
    }
    const float g = decay[(int)(bh % H)];
    float4 vv = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col) {
        vv.x = load_elem<BF16>(v, bh * dv + j);
        vv.y = load_elem<BF16>(v, bh * dv + j + 1);
        vv.z = load_elem<BF16>(v, bh * dv + j + 2);
        vv.w = load_elem<BF16>(v, bh * dv + j + 3);
    }
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        const float kr = ks[warp * RW + i], qr = qs[warp * RW + i];
        float4 t;
        t.x = fmaf(g, s[i].x, kr * vv.x);
        t.y = fmaf(g, s[i].y, kr * vv.y);
        t.z = fmaf(g, s[i].z, kr * vv.z);
        t.w = fmaf(g, s[i].w, kr * vv.w);
        if (col && warp * RW + i < r) st_stream(Sr + (size_t)i * dv4, t);
        acc.x = fmaf(qr, t.x, acc.x);
        acc.y = fmaf(qr, t.y, acc.y);
        acc.z = fmaf(qr, t.z, acc.z);
        acc.w = fmaf(qr, t.w, acc.w);
    }
    part[warp][lane] = acc;
    __syncthreads();
    if (tid < 128 && c0 + tid < dv) {
        const float *p = reinterpret_cast<const float *>(part);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) sum += p[w * 128 + tid];
        store_elem<BF16>(y, bh * dv + c0 + tid, sum * scale);
    }
}

template <bool BF16>
cudaError_t launch_dec(const void *q, const void *k, const void *v, const float *decay, float *S, int BH, int H, int r,
                       int dv, float scale, void *y, cudaStream_t stream)
{
    const dim3 grid(BH, (dv + 127) / 128);
    if (r <= 64) decay_decode_kernel<BF16, 8><<<grid, 256, 0, stream>>>(q, k, v, decay, S, H, r, dv, scale, y);
    else if (r <= 128) decay_decode_kernel<BF16, 16><<<grid, 256, 0, stream>>>(q, k, v, decay, S, H, r, dv, scale, y);
    else decay_decode_kernel<BF16, 32><<<grid, 256, 0, stream>>>(q, k, v, decay, S, H, r, dv, scale, y);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decay_rec(const DecaySweep *sweeps, int count, const DecayArgs &a, bool bf16, int B,
                             cudaStream_t stream)
{
    RecArgs r;
    r.d = a;
    int rows = 0, tiles = 0;
    for (int i = 0; i < 3; ++i) {
        r.tiles[i] = 0;
        if (i >= count) continue;
        r.sw[i] = sweeps[i];
        r.tiles[i] = (sweeps[i].n + kRecCols - 1) / kRecCols;
        tiles += r.tiles[i];
        rows = sweeps[i].ra > rows ? sweeps[i].ra : rows;
    }
    const dim3 grid(tiles, a.H, B);
    return bf16 ? launch_rec<true>(r, rows, grid, stream) : launch_rec<false>(r, rows, grid, stream);
}

cudaError_t launch_decay_decode(const void *q, const void *k, const void *v, bool bf16, const float *decay, float *S,
                                int B, int H, int r, int dv, float scale, void *y, cudaStream_t stream)
{
    return bf16 ? launch_dec<true>(q, k, v, decay, S, B * H, H, r, dv, scale, y, stream)
                : launch_dec<false>(q, k, v, decay, S, B * H, H, r, dv, scale, y, stream);
}

}  // namespace la
