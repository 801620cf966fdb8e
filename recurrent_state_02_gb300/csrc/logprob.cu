// logprob.cu -- scoring given tokens: log-probabilities, entropy and best alternatives of rows of logits, and
// the gradient of the first two.
//
//     lse = log sum_v exp x_v,   logprob = x_token - lse,   H = lse - sum_v p_v x_v,   p_v = exp(x_v - lse)
//     dL/dx_v = dlogprob (1[v = token] - p_v) - dH p_v (log p_v + H)

#include "gdelta.h"
#include "sm103_ptx.cuh"

#include <cuda_bf16.h>

namespace la {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.402823466e38f;

// 2^x, relative error about 2^-22 (results below 2^-126 are 0: nothing next to the maximum's 1)
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Order-preserving map of a float (not NaN) to unsigned; -0 counts as +0.
__device__ __forceinline__ uint32_t order_f32(float x)
{
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unorder_f32(uint32_t o)
{
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
// Keys that order by value, then by lower index; 0 is none.
__device__ __forceinline__ unsigned long long make_key(float x, int i)
{
    return (static_cast<unsigned long long>(order_f32(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ unsigned long long warp_max(unsigned long long k)
{
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(k >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
    return (static_cast<unsigned long long>(hi) << 32) | lo;
}

template <typename T>
__device__ __forceinline__ T *in_cta(T *p, uint32_t rank)
{
    uint64_t out;
    asm volatile("mapa.u64 %0, %1, %2;" : "=l"(out) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
    return reinterpret_cast<T *>(out);
}
__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint4 ld_once(const uint4 *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <bool BF16>
__device__ __forceinline__ void widen(uint4 w, float *x)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        } else {
            x[i] = __uint_as_float(u[i]);
        }
    }
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// x - m of the two BF16 values in w, without widening them first
__device__ __forceinline__ float2 minus_bf16x2(uint32_t w, float m)
{
    float2 d;
    asm("{\n\t.reg .b16 a, b, one;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "mov.b16 one, 0x3F80;\n\t"
        "fma.rn.f32.bf16 %0, a, one, %3;\n\t"
        "fma.rn.f32.bf16 %1, b, one, %3;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "r"(w), "f"(-m));
    return d;
}
// Logits below this (a BF16 number) count as this in the sums, so that x - m stays finite and a masked one's term is 0; what a
// lane with nothing above it, or with a maximum as far up, has seen is summed again with care.
constexpr float kFloor = -1.171875f * 0x1p126f;  // -9.97e37

// Largest of a granule's values (a NaN among them does not show), and its values, at least `floor`, less m.
template <bool BF16>
__device__ __forceinline__ float granule_max(uint4 w)
{
    if (BF16) {
        uint32_t a, b, c;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(w.x), "r"(w.y));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(w.z), "r"(w.w));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
        return fmaxf(bf16_lo(c), bf16_hi(c));
    }
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
}
template <bool BF16>
__device__ __forceinline__ void granule_minus(uint4 w, float m, float floor, float2 *d)
{
    if (BF16) {
        const uint32_t f = pack_bf16x2(floor, floor);
        d[0] = minus_bf16x2(max_nan_bf16x2(w.x, f), m);
        d[1] = minus_bf16x2(max_nan_bf16x2(w.y, f), m);
        d[2] = minus_bf16x2(max_nan_bf16x2(w.z, f), m);
        d[3] = minus_bf16x2(max_nan_bf16x2(w.w, f), m);
    } else {
        const float2 minus = make_float2(-m, -m);
        d[0] = __fadd2_rn(make_float2(max_nan(__uint_as_float(w.x), floor), max_nan(__uint_as_float(w.y), floor)), minus);
        d[1] = __fadd2_rn(make_float2(max_nan(__uint_as_float(w.z), floor), max_nan(__uint_as_float(w.w), floor)), minus);
    }
}

template <bool BF16>
__device__ __forceinline__ float load_elem(const void *p, long long i)
{
    return BF16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16) : static_cast<const float *>(p)[i];
}

// Granule `lane` of block `blk` of a row of V elements: 16 bytes of an aligned row, else elements 32 apart
// (element e of the granule is element granule_first + e * ES of the row).  -infinity past the row's end.
template <bool BF16, bool ALIGNED>
__device__ __forceinline__ uint4 load_granule(const void *row, int blk, int lane, int V)
{
    constexpr int GE = BF16 ? 8 : 4, ES = ALIGNED ? 1 : 32;
    const int i0 = ALIGNED ? (blk * 32 + lane) * GE : blk * 32 * GE + lane;
    if (ALIGNED && i0 + GE <= V) return ld_once(reinterpret_cast<const uint4 *>(row) + (blk * 32 + lane));
    uint32_t x[GE], w[4];
#pragma unroll
    for (int e = 0; e < GE; ++e) {
        x[e] = BF16 ? 0xff80u : 0xff800000u;
        if (i0 + ES * e < V)
            x[e] = BF16 ? static_cast<const uint16_t *>(row)[i0 + ES * e] : static_cast<const uint32_t *>(row)[i0 + ES * e];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = BF16 ? x[2 * j] | x[2 * j + 1] << 16 : x[j];
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// ------------------------------------------------------------------- scoring
// One cluster of CS CTAs of 8 warps per row, one pass over the row: every lane carries a running maximum m, the sum
// s of 2^a and the sum w of a 2^a, a = (x - m) log2 e, from which lse and the entropy follow.  The alternatives come from
// maxima that the pass forms anyway: a lane's maximum of four blocks of 32 granules joins its warp's, an entry covers one such
// group or 2^shift of them, and the entries are gathered to 64 group maxima per CTA, whose top-th largest bounds the top-th
// best from below.  Only the groups that reach it are read again, by all warps alike (about as many as there are alternatives, out of
// L2), and what reaches it is ranked by counting what is better.
// Bound by exponentials and issue slots beside HBM: N = 2048, V = 131072, top 8, BF16 94 us (5.7 TB/s; 82 without alternatives,
// 6.5 TB/s); 5 CTAs per SM hold 48 registers (one instance spills 12 bytes; 6 CTAs spill more and are slower).  A row's end costs its CTA
// about 4 us with alternatives, which short rows feel: N = 8192, V = 32000, top 8 133 us, without 83.  (Each warp reading its own
// groups again and one warp picking the best one by one: 98 and 143.)
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kEntries = 64;       // maxima per warp: an entry covers 2^shift of its groups of 4 blocks
constexpr int kGroups = 64;        // of a CTA's entries: 8 per warp
constexpr int kCand = 512;

struct ScoreSmem {
    uint32_t entry[kWarps][kEntries];              // order_f32 of the maximum (0: no logit above -infinity)
    uint32_t group[kGroups];
    unsigned long long cand[kCand];
    unsigned long long best[kMaxTop];              // this CTA's
    uint16_t again[kWarps * kEntries];             // the entries that reach the bound: warp, entry
    float m[kWarps], s[kWarps], w[kWarps];
    float cm, cs, cw;                              // the CTA's
    uint32_t thr;                                  // what an alternative reaches at least
    int count, entries;
};

// Merges (m, s, w) of two parts.
__device__ __forceinline__ void merge(float &m, float &s, float &w, float m2, float s2, float w2)
{
    const float mm = fmaxf(m, m2);
    // (an empty part has s = 0 and m = kLowest: its difference must not become 0 * infinity)
    const float d1 = fmaxf((m - mm) * kLog2e, -400.f), d2 = fmaxf((m2 - mm) * kLog2e, -400.f);
    const float c1 = ex2(d1), c2 = ex2(d2);
    w = (w + s * d1) * c1 + (w2 + s2 * d2) * c2;
    s = s * c1 + s2 * c2;
    m = mm;
}

template <bool BF16, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 5)
token_logprobs_kernel(const LogprobArgs args)
{
    constexpr int GE = BF16 ? 8 : 4, ES = ALIGNED ? 1 : 32, U = 4;
    __shared__ ScoreSmem sm;
    const int V = args.V, top = args.top;
    const uint32_t rank = blockIdx.x, cs = gridDim.x;   // the cluster spans the grid's x axis
    const long long n = blockIdx.y + (long long)gridDim.y * blockIdx.z;
    if (n >= args.N) return;                            // (the whole cluster)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int token = args.tokens[n];
    if (token < 0 || token >= V) {
        if (rank == 0) {
            if (tid == 0) {
                args.logprobs[n] = 0.f;
                if (args.entropy) args.entropy[n] = 0.f;
                if (args.lse) args.lse[n] = 0.f;
                if (token >= V) atomicExch(args.status, kStatusShape);
            }
            if (tid < top) args.top_logprobs[n * top + tid] = -INFINITY, args.top_tokens[n * top + tid] = -1;
        }
        return;
    }
    const unsigned char *row = static_cast<const unsigned char *>(args.logits) + n * args.row_stride * (BF16 ? 2 : 4);
    const float x_token = rank == 0 && tid == 0 ? load_elem<BF16>(row, token) : 0.f;
    const int blocks = (V + 32 * GE - 1) / (32 * GE);
    const int nw = kWarps * cs, gw = rank * kWarps + warp;
    int shift = 0;
    while (((blocks + U * nw - 1) / (U * nw) - 1) >> shift >= kEntries) ++shift;
    if (top) {
        sm.entry[warp][lane] = sm.entry[warp][lane + 32] = 0;
        if (tid == 0) sm.count = sm.entries = 0;
        if (tid < kMaxTop) sm.best[tid] = 0;
        __syncwarp();
    }
    float m = kFloor, s = 0.f, w = 0.f;
    // takes U granules of this lane into m, s and w, and their maximum into the group's entry
    auto take = [&](const uint4 (&raw)[U], int group) {
        float mx = granule_max<BF16>(raw[0]);
#pragma unroll
        for (int u = 1; u < U; ++u) mx = fmaxf(mx, granule_max<BF16>(raw[u]));   // (a NaN reaches the sums below)
        if (mx > m) {
            const float d = fmaxf((m - mx) * kLog2e, -400.f);
            w = (w + s * d) * ex2(d);
            s *= ex2(d);
            m = mx;
        }
        const float2 l2 = make_float2(kLog2e, kLog2e);
        float2 t = make_float2(0.f, 0.f), tw = t;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 a[GE / 2];
            granule_minus<BF16>(raw[u], m, kFloor, a);
#pragma unroll
            for (int e = 0; e < GE / 2; ++e) {
                a[e] = __fmul2_rn(a[e], l2);
                const float2 p = make_float2(ex2(a[e].x), ex2(a[e].y));
                t = __fadd2_rn(t, p);
                tw = __ffma2_rn(a[e], p, tw);
            }
        }
        s += t.x + t.y;
        w += tw.x + tw.y;
        if (top) {
            const uint32_t o = __reduce_max_sync(0xffffffffu, mx > -INFINITY ? order_f32(mx) : 0u);
            uint32_t &en = sm.entry[warp][group >> shift];
            if (lane == 0 && o > en) en = o;
        }
    };
    int blk = gw, group = 0;
    // (whole groups of aligned rows need no look at the row's end)
    for (; ALIGNED && (long long)(blk + (U - 1) * nw + 1) * 32 * GE <= V; blk += U * nw, ++group) {
        uint4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = ld_once(reinterpret_cast<const uint4 *>(row) + ((blk + u * nw) * 32 + lane));
        take(raw, group);
    }
    for (; blk < blocks; blk += U * nw, ++group) {
        uint4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = load_granule<BF16, ALIGNED>(row, blk + u * nw, lane, V);   // (-infinity behind the row)
        take(raw, group);
    }
    // (masks and lowest values only, or none at all, up to a whole row of them; a maximum of +infinity stays: its sums are not
    // numbers)
    const bool odd = m <= kFloor || (m >= -kFloor && m < INFINITY);
    if (__any_sync(0xffffffffu, odd)) {
        if (odd) {
            m = kLowest, s = w = 0.f;
            for (int blk = gw; blk < blocks; blk += nw) {
                float x[GE];
                widen<BF16>(load_granule<BF16, ALIGNED>(row, blk, lane, V), x);
#pragma unroll
                for (int e = 0; e < GE; ++e) {
                    if (x[e] > -INFINITY) merge(m, s, w, x[e], 1.f, 0.f);
                    if (x[e] != x[e]) s = x[e];
                }
            }
        }
        __syncwarp();
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o),
                    w2 = __shfl_xor_sync(0xffffffffu, w, o);
        merge(m, s, w, m2, s2, w2);
    }
    if (lane == 0) sm.m[warp] = m, sm.s[warp] = s, sm.w[warp] = w;
    if (top) {
        __syncwarp();
        if (lane < 8) {
            uint32_t best = 0;
#pragma unroll
            for (int e = 0; e < kEntries; e += 8) best = max(best, sm.entry[warp][e + lane]);
            sm.group[warp * 8 + lane] = best;
        }
    }
    __syncthreads();
    if (warp == 0) {
        m = lane < kWarps ? sm.m[lane] : kLowest, s = lane < kWarps ? sm.s[lane] : 0.f, w = lane < kWarps ? sm.w[lane] : 0.f;
#pragma unroll
        for (int o = kWarps / 2; o; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o),
                        w2 = __shfl_xor_sync(0xffffffffu, w, o);
            merge(m, s, w, m2, s2, w2);
        }
        if (lane == 0) sm.cm = m, sm.cs = s, sm.cw = w;
    }
    if (top) {
        // the top-th largest group maximum: four lanes rank a group, a warp its own eight
        const int g = warp * 8 + (lane >> 2);
        const uint32_t mine = sm.group[g];
        int above = 0;
#pragma unroll
        for (int i = 0; i < kGroups / 4; ++i) {
            const int o = i * 4 + (lane & 3);
            const uint32_t v = sm.group[o];
            above += v > mine || (v == mine && o < g);
        }
        above += __shfl_xor_sync(0xffffffffu, above, 1);
        above += __shfl_xor_sync(0xffffffffu, above, 2);
        if (above == top - 1) sm.thr = max(1u, mine);
        __syncthreads();
        const uint32_t thr = sm.thr;
        // the entries that reach it, as a list: their blocks are read again by all warps alike
        for (int e = lane; e < kEntries; e += 32)
            if (sm.entry[warp][e] >= thr) sm.again[atomicAdd(&sm.entries, 1)] = (uint16_t)(warp * kEntries + e);
        __syncthreads();
        const int per = U << shift, total = sm.entries * per;        // (blocks behind the row are -infinity)
        for (int i0 = U * warp; i0 < total; i0 += U * kWarps) {
            // (U divides what an entry covers)
            const int from = sm.again[i0 / per], b0 = (int)rank * kWarps + from / kEntries + ((from % kEntries) * per + i0 % per) * nw;
            uint4 raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) raw[u] = load_granule<BF16, ALIGNED>(row, b0 + u * nw, lane, V);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float mx = granule_max<BF16>(raw[u]);
                if (!(mx > -INFINITY && order_f32(mx) >= thr)) continue;
                float x[GE];
                widen<BF16>(raw[u], x);
#pragma unroll
                for (int i = 0; i < GE; ++i)
                    if (x[i] > -INFINITY && order_f32(x[i]) >= thr) {
                        const int at = atomicAdd(&sm.count, 1);
                        if (at < kCand)
                            sm.cand[at] = make_key(x[i], (ALIGNED ? ((b0 + u * nw) * 32 + lane) * GE : (b0 + u * nw) * 32 * GE + lane) + i * ES);
                    }
            }
        }
        __syncthreads();
        const int count = sm.count;
        if (count > kCand) {
            // many equal logits: every warp keeps the best of its blocks, lane r the r-th, and no order of the
            // pushes matters (sorted by value and index)
            __syncthreads();
            unsigned long long mine = 0;
            for (int blk = gw; blk < blocks; blk += nw) {
                float x[GE];
                widen<BF16>(load_granule<BF16, ALIGNED>(row, blk, lane, V), x);
#pragma unroll 1
                for (int i = 0; i < GE; ++i) {
                    float xi = x[0];
#pragma unroll
                    for (int f = 1; f < GE; ++f) xi = i == f ? x[f] : xi;
                    unsigned long long key = xi > -INFINITY && order_f32(xi) >= thr
                                                 ? make_key(xi, (ALIGNED ? (blk * 32 + lane) * GE : blk * 32 * GE + lane) + i * ES)
                                                 : 0;
                    const unsigned long long least = __shfl_sync(0xffffffffu, mine, top - 1);
                    if (key <= least) key = 0;
                    while (__any_sync(0xffffffffu, key != 0)) {
                        const unsigned long long k = warp_max(key);
                        if (key == k) key = 0;
                        const unsigned long long up = __shfl_up_sync(0xffffffffu, mine, 1);
                        if (k > mine) mine = lane == 0 || up > k ? k : up;
                        if (key <= __shfl_sync(0xffffffffu, mine, top - 1)) key = 0;
                    }
                }
            }
            if (lane < top) sm.cand[warp * top + lane] = mine;
            __syncthreads();
        }
        // a candidate's place is how many are better
        const int have = count > kCand ? kWarps * top : count;
        for (int i = tid; i < have; i += kThreads) {
            const unsigned long long mine = sm.cand[i];
            int place = 0;
            for (int j = 0; j < have && place < top; ++j) place += sm.cand[j] > mine;
            if (mine && place < top) sm.best[place] = mine;
        }
    }
    if (cs > 1) cluster_sync_all();
    else __syncthreads();
    if (rank == 0 && warp == 0) {
        // (every lane forms the same row sums)
        m = sm.cm, s = sm.cs, w = sm.cw;
        for (uint32_t c = 1; c < cs; ++c) {
            ScoreSmem *at = in_cta(&sm, c);
            merge(m, s, w, at->cm, at->cs, at->cw);
        }
        const float lg = logf(s);
        const bool fine = s > 0.f && m < INFINITY, empty = s == 0.f;   // (a NaN is neither)
        const float nan = __int_as_float(0x7fffffff);
        if (lane == 0) {
            args.logprobs[n] = fine ? (x_token - m) - lg : empty ? -INFINITY : nan;
            if (args.entropy) args.entropy[n] = fine ? fmaxf(lg - kLn2 * (w / s), 0.f) : empty ? 0.f : nan;
            if (args.lse) args.lse[n] = fine ? m + lg : empty ? -INFINITY : nan;
        }
        // the best of the CTAs' best: lane r ends with the r-th
        unsigned long long mine = 0;
        if (top && cs == 1) {
            mine = lane < top ? sm.best[lane] : 0;
        } else if (top) {
            unsigned long long k[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) k[i] = i < (int)cs && lane < top ? in_cta(&sm, i)->best[lane] : 0;
#pragma unroll 1
            for (int r = 0; r < top; ++r) {
                unsigned long long best = k[0];
#pragma unroll
                for (int i = 1; i < 8; ++i) best = k[i] > best ? k[i] : best;
                best = warp_max(best);
                if (lane == r) mine = best;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (k[i] == best) k[i] = 0;
            }
        }
        if (lane < top) {
            const bool have = fine && mine != 0;
            args.top_logprobs[n * top + lane] = have ? (unorder_f32((uint32_t)(mine >> 32)) - m) - lg : -INFINITY;
            args.top_tokens[n * top + lane] = have ? (int)(0xffffffffu - (uint32_t)mine) : -1;
        }
    }
    if (cs > 1) cluster_sync_all();       // a CTA's shared memory stays until it has been read
}

template <bool BF16, bool ALIGNED>
cudaError_t launch_score(const LogprobArgs &a, int cs, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg{};
    const long long rows = a.N;
    const unsigned ny = (unsigned)(rows < 65535 ? rows : 65535);
    cfg.gridDim = dim3(cs, ny, (unsigned)((rows + ny - 1) / ny));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cs, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<BF16, ALIGNED>, a);
}

// ------------------------------------------------------------------ gradient
// One CTA per row and 2048 granules of 16 bytes; each is read, turned into its gradient and written, eight in flight per
// thread.  Rows without a token get zeros and are not read.  Bound by HBM: N = 8192, V = 32000, BF16 167 us, 6.1 TB/s.
// lse is FP32, so p carries half a step of it, 2^-18 at 64 to 128.  Rows further off than that (one huge value, as a mask
// of the type's lowest) have their maximum and sum formed again, by a single CTA, which then does the whole row.
constexpr int kGradThreads = 256, kGradU = 8;
constexpr float kFarLse = 128.f;

template <bool BF16, bool ALIGNED>
__global__ void __launch_bounds__(kGradThreads)
token_logprobs_backward_kernel(const LogprobGradArgs args, int slices)
{
    constexpr int GE = BF16 ? 8 : 4, ES = ALIGNED ? 1 : 32, kWarpsG = kGradThreads / 32;
    __shared__ float part[2][kWarpsG];
    const int V = args.V;
    const long long n = blockIdx.x / slices;
    const int slice = blockIdx.x % slices, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int token = args.tokens[n];
    const unsigned char *row = static_cast<const unsigned char *>(args.logits) + n * args.row_stride * (BF16 ? 2 : 4);
    unsigned char *out = static_cast<unsigned char *>(args.dlogits) + n * args.grad_stride * (BF16 ? 2 : 4);
    const bool skip = token < 0 || token >= V;
    if (token >= V && tid == 0) atomicExch(args.status, kStatusShape);
    const int blocks = (V + 32 * GE - 1) / (32 * GE);
    uint4 raw[kGradU];
    // this warp's u-th block of 32 granules of a slice
    auto block_of = [&](int sl, int u) { return (sl * kGradU + u) * kWarpsG + warp; };
    auto load = [&](int sl) {
#pragma unroll
        for (int u = 0; u < kGradU; ++u)
            if (block_of(sl, u) < blocks) raw[u] = load_granule<BF16, ALIGNED>(row, block_of(sl, u), lane, V);
    };
    if (!skip) load(slice);
    const float lse = skip ? 0.f : args.lse[n], dlp = skip ? 0.f : args.dlogprobs[n];
    const float dH = skip || !args.dentropy ? 0.f : args.dentropy[n], H = dH != 0.f ? args.entropy[n] : 0.f;
    const bool zero = skip || lse == -INFINITY;
    // log p_v = (x_v - m) - lg
    float m = lse, lg = 0.f;
    const bool far = !zero && fabsf(lse) >= kFarLse;
    if (far) {
        if (slice) return;
        float s = 0.f, w = 0.f;
        m = kLowest;
        for (int blk = warp; blk < blocks; blk += kWarpsG) {
            float x[GE];
            widen<BF16>(load_granule<BF16, ALIGNED>(row, blk, lane, V), x);
#pragma unroll
            for (int e = 0; e < GE; ++e)
                if (x[e] > -INFINITY) merge(m, s, w, x[e], 1.f, 0.f);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
            merge(m, s, w, m2, s2, 0.f);
        }
        if (lane == 0) part[0][warp] = m, part[1][warp] = s;
        __syncthreads();
        m = kLowest, s = 0.f;
        for (int i = 0; i < kWarpsG; ++i) merge(m, s, w, part[0][i], part[1][i], 0.f);
        lg = logf(s);
    }
    // g = -p (c0 + dH log p), c0 = dlp + dH H
    const float c0 = fmaf(dH, H, dlp);
    const int end = far ? slices : slice + 1;
    for (int sl = slice; sl < end; ++sl) {
        if (far) load(sl);
#pragma unroll
        for (int u = 0; u < kGradU; ++u) {
            const int blk = block_of(sl, u);
            if (blk >= blocks) break;
            const int i0 = ALIGNED ? (blk * 32 + lane) * GE : blk * 32 * GE + lane;
            float gr[GE];
            if (zero) {
#pragma unroll
                for (int e = 0; e < GE; ++e) gr[e] = 0.f;
            } else {
                // (log p of at least -200, where p is 0: a masked logit's is not infinite)
                float2 lp[GE / 2];
                if (!far) {
                    granule_minus<BF16>(raw[u], m, m - 200.f, lp);
                } else {
                    float x[GE];
                    widen<BF16>(raw[u], x);
#pragma unroll
                    for (int e = 0; e < GE / 2; ++e)
                        lp[e] = make_float2(max_nan((x[2 * e] - m) - lg, -200.f), max_nan((x[2 * e + 1] - m) - lg, -200.f));
                }
#pragma unroll
                for (int e = 0; e < GE / 2; ++e) {
                    const float2 a = __fmul2_rn(lp[e], make_float2(kLog2e, kLog2e));
                    const float2 g = __fmul2_rn(make_float2(-ex2(a.x), -ex2(a.y)), __ffma2_rn(make_float2(dH, dH), lp[e], make_float2(c0, c0)));
                    gr[2 * e] = g.x, gr[2 * e + 1] = g.y;
                }
                const int at = token - i0;
                if (at >= 0 && at < GE * ES && at % ES == 0) {
#pragma unroll
                    for (int e = 0; e < GE; ++e)
                        if (at == e * ES) gr[e] += dlp;
                }
            }
            if (ALIGNED && i0 + GE <= V) {
                uint4 o;
                if (BF16) o = make_uint4(pack_bf16x2(gr[0], gr[1]), pack_bf16x2(gr[2], gr[3]), pack_bf16x2(gr[4 % GE], gr[5 % GE]),
                                         pack_bf16x2(gr[6 % GE], gr[7 % GE]));
                else o = make_uint4(__float_as_uint(gr[0]), __float_as_uint(gr[1]), __float_as_uint(gr[2]), __float_as_uint(gr[3]));
                reinterpret_cast<uint4 *>(out)[blk * 32 + lane] = o;
            } else {
#pragma unroll
                for (int e = 0; e < GE; ++e)
                    if (i0 + e * ES < V) {
                        if (BF16) reinterpret_cast<uint16_t *>(out)[i0 + e * ES] = (uint16_t)(pack_bf16x2(gr[e], 0.f) & 0xffffu);
                        else reinterpret_cast<float *>(out)[i0 + e * ES] = gr[e];
                    }
            }
        }
    }
}

bool rows_aligned(const void *p, long long stride, bool bf16)
{
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (stride * (bf16 ? 2 : 4)) % 16 == 0;
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs &a, bool bf16, int sms, cudaStream_t stream)
{
    // a row is spread over up to 8 CTAs until the device has about two per SM
    int cs = 1;
    while (cs < 8 && (long long)a.N * cs < 2LL * sms) cs *= 2;
    const bool al = a.N == 1 ? rows_aligned(a.logits, 0, bf16) : rows_aligned(a.logits, a.row_stride, bf16);
    if (bf16) return al ? launch_score<true, true>(a, cs, stream) : launch_score<true, false>(a, cs, stream);
    return al ? launch_score<false, true>(a, cs, stream) : launch_score<false, false>(a, cs, stream);
}

cudaError_t launch_token_logprobs_backward(const LogprobGradArgs &a, bool bf16, int, cudaStream_t stream)
{
    const int ge = bf16 ? 8 : 4, per = kGradThreads * kGradU * ge, slices = (a.V + per - 1) / per;
    const unsigned grid = (unsigned)((long long)a.N * slices);
    const bool al = (a.N == 1 ? rows_aligned(a.logits, 0, bf16) : rows_aligned(a.logits, a.row_stride, bf16)) &&
                    (a.N == 1 ? rows_aligned(a.dlogits, 0, bf16) : rows_aligned(a.dlogits, a.grad_stride, bf16));
    if (bf16) {
        if (al) token_logprobs_backward_kernel<true, true><<<grid, kGradThreads, 0, stream>>>(a, slices);
        else token_logprobs_backward_kernel<true, false><<<grid, kGradThreads, 0, stream>>>(a, slices);
    } else {
        if (al) token_logprobs_backward_kernel<false, true><<<grid, kGradThreads, 0, stream>>>(a, slices);
        else token_logprobs_backward_kernel<false, false><<<grid, kGradThreads, 0, stream>>>(a, slices);
    }
    return cudaGetLastError();
}

}  // namespace la
