// beam.cu -- what a beam search does between two decode steps: choose the best
// K of a request's K beams x V tokens, and move the beams' states after the choice.

#include "decay.h"
#include "launch_rules.h"
#include "sm103_ptx.cuh"

#include <cuda_bf16.h>

namespace la {
namespace {

// ------------------------------------------------------------- beam select
// Candidate (k, v) of a request scores  score_k + x_kv - lse_k,  lse_k = log sum_v
// exp x_kv.  Within a beam the candidates rank as its logits do, so one pass over
// a row yields both its log-sum-exp (running maximum and sum per lane) and its
// best K logits; K * K finalists then settle the request.
//
// One cluster of CS CTAs of 16 warps per request.  Warp gw of the cluster's 16 CS
// takes part gw / K of row gw % K: 512-byte blocks, every (parts)-th one.  It pushes the logits
// that may be among the row's K best into a buffer of its own, as 64-bit keys that order by
// logit, then by lower index, and keeps the K best of a full buffer; the K-th of them, at
// first the K-th largest of the lanes' maxima, is what a logit has to beat, so a block
// without one costs a vote.
// After the cluster barrier warp w of CTA c merges the parts of row c + CS w (over
// distributed shared memory) and leaves the row's K keys and its lse in CTA 0;
// after the second one a warp of CTA 0 picks the request's K best by the scores
// in 64 bits, one head per row.
//
// Bound by instructions, not by HBM: B64 K4 V131072 BF16 takes 33 us, the 67 MB would
// take 10 at the copy bandwidth; 7 us are the launch, the barriers and the merge (V = 100).
constexpr int kSelWarps = 16, kSelThreads = 32 * kSelWarps;

constexpr int kSelBuf = 128;    // keys of a warp's buffer

struct SelSmem {
    unsigned long long keys[kSelWarps][kSelBuf];          // each warp's candidates; at the end its K best, best first (0: none)
    float m[kSelWarps], s[kSelWarps];                     // running maximum and sum of its part
    int count[kSelWarps];                                 // keys in its buffer
    unsigned long long bound[kMaxBeams];                  // a K-th key of some part of a row, which all its warps share
    // CTA 0 only: the rows' best, and their lse as a maximum and the logarithm of the sum next to it (a maximum of
    // 1e17 or more, a mask of the type's lowest value for one, would swallow the logarithm)
    unsigned long long row_keys[kMaxBeams][kMaxBeams];
    float row_max[kMaxBeams];
    double row_log[kMaxBeams];
};

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
__device__ __forceinline__ unsigned long long order_f64(double x)
{
    const unsigned long long u = __double_as_longlong(x + 0.0);
    return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ unsigned long long make_key(float x, int i)
{
    return (static_cast<unsigned long long>(order_f32(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ int key_index(unsigned long long k) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)); }
__device__ __forceinline__ float key_value(unsigned long long k) { return unorder_f32(static_cast<uint32_t>(k >> 32)); }

// Largest key of the warp (every lane gets it).
__device__ __forceinline__ unsigned long long warp_max(unsigned long long k)
{
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(k >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
    return (static_cast<unsigned long long>(hi) << 32) | lo;
}

// Distributed shared memory: the generic address of `p` in CTA `rank` of the cluster.
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
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// A lane's granule by single elements i, i + ES, .. of the row (0 past its end), packed like the 16 bytes of a whole
// one: of rows that do not all start on 16-byte boundaries (ES = 32), or what is left of an aligned row (ES = 1).
template <bool BF16, int ES>
__device__ __forceinline__ uint4 load_elements(const void *row, int i, int V)
{
    constexpr int GE = BF16 ? 8 : 4;
    uint32_t x[GE], w[4];
#pragma unroll
    for (int e = 0; e < GE; ++e) {
        x[e] = 0;
        if (i + ES * e < V)
            x[e] = BF16 ? reinterpret_cast<const uint16_t *>(row)[i + ES * e] : reinterpret_cast<const uint32_t *>(row)[i + ES * e];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = BF16 ? x[2 * j] | x[2 * j + 1] << 16 : x[j];
    return make_uint4(w[0], w[1], w[2], w[3]);
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

constexpr float kLog2e = 1.4426950408889634f;

// 2^x, relative error about 2^-22 (results below 2^-126 are 0: nothing next to the maximum's 1)
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ALIGNED: every row starts on a 16-byte boundary, and a lane's granule is 16 bytes of it; else it is elements 32 apart.
// (Which element goes to which lane depends on its index alone, so equal rows have equal sums.)
// REST: a granule may be left over at the end of an aligned row (an instance of its own, as even an untaken branch costs
// the loop registers: B64 K4 V131072 30.4 us with it, 29.8 without).
template <bool BF16, bool ALIGNED, bool REST>
__global__ void __launch_bounds__(kSelThreads, 2)
beam_select_kernel(const BeamSelectArgs args)
{
    constexpr int GE = BF16 ? 8 : 4;       // elements of a 16-byte granule
    constexpr int U = 4;                   // granules in flight per lane
    constexpr int ES = ALIGNED ? 1 : 32;   // from one element of a granule to the next
    __shared__ SelSmem sm;
    const int K = args.K, V = args.V;
    const uint32_t rank = blockIdx.x, cs = gridDim.x;   // the cluster spans the grid's x axis
    const int b = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nw = kSelWarps * cs;
    if (threadIdx.x < kMaxBeams) sm.bound[threadIdx.x] = 0;
    // what phase 3 needs, in flight from the start
    const bool picks = rank == 0 && warp == 0 && lane < K;
    const size_t bk = (size_t)b * K;
    const float score_f = picks ? args.scores[bk + lane] : 0.f;
    const bool ended = picks && args.done && args.done[bk + lane];
    __syncthreads();
    {
        // phase 1: this warp's part of one row
        const int gw = rank * kSelWarps + warp;
        // (every row has the same number of parts, so that equal rows have equal sums to the last bit and tie;
        // warps left over are idle)
        const int k = gw % K, part = gw / K, parts = nw / K;
        const bool skip = part >= parts || (args.done && args.done[(size_t)b * K + k]);
        const unsigned char *row = reinterpret_cast<const unsigned char *>(args.logits) +
                                   ((long long)b * K + k) * args.row_stride * (BF16 ? 2 : 4);
        const int granules = ALIGNED ? (V + GE - 1) / GE : (V + 32 * GE - 1) / (32 * GE) * 32;
        const int whole = REST ? whole_granules(V, GE) : granules;
        float m = -3.402823466e38f, s = 0.f;
        unsigned long long thr = 0;      // what a key has to beat
        float thr_x = -INFINITY;         // its logit
        bool seeded = false;
        int count = 0;                   // keys in the buffer
        unsigned long long *buf = sm.keys[warp];
        // keeps the K best of the buffer, sorted
        auto keep_best = [&]() {
            __syncwarp();
            unsigned long long k0 = lane < count ? buf[lane] : 0, mine = 0;
            if (count <= 32) {
#pragma unroll 1
                for (int r = 0; r < K; ++r) {
                    const unsigned long long best = warp_max(k0);
                    if (lane == r) mine = best;
                    if (k0 == best) k0 = 0;
                }
            } else {
                unsigned long long k1 = lane + 32 < count ? buf[lane + 32] : 0, k2 = lane + 64 < count ? buf[lane + 64] : 0,
                                   k3 = lane + 96 < count ? buf[lane + 96] : 0;
#pragma unroll 1
                for (int r = 0; r < K; ++r) {
                    const unsigned long long a = k0 > k1 ? k0 : k1, c = k2 > k3 ? k2 : k3;
                    const unsigned long long best = warp_max(a > c ? a : c);
                    if (lane == r) mine = best;
                    if (k0 == best) k0 = 0;
                    if (k1 == best) k1 = 0;
                    if (k2 == best) k2 = 0;
                    if (k3 == best) k3 = 0;
                }
            }
            if (lane < K) buf[lane] = mine;
            if (count >= K) {
                thr = __shfl_sync(0xffffffffu, mine, K - 1);
                thr_x = key_value(thr);
                count = K;
                if (lane == 0) sm.count[warp] = K, atomicMax(&sm.bound[k], thr);
            }
            __syncwarp();
        };
        // takes a granule into the running maximum and sum; returns its maximum
        auto sum_up = [&](uint4 raw, int i0) -> float {
            float x[GE];
            widen<BF16>(raw, x);
            if (i0 + (GE - 1) * ES >= V) {
#pragma unroll
                for (int e = 0; e < GE; ++e)
                    if (i0 + e * ES >= V) x[e] = -INFINITY;
            }
            float mx = x[0];
#pragma unroll
            for (int e = 1; e < GE; ++e) mx = fmaxf(mx, x[e]);   // (a NaN reaches the sum below)
            if (mx > m) {
                s *= ex2((m - mx) * kLog2e);
                m = mx;
            }
            const float2 minus = make_float2(-m, -m), l2 = make_float2(kLog2e, kLog2e);
            float2 t = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < GE; e += 2) {
                const float2 a = __fmul2_rn(__fadd2_rn(make_float2(x[e], x[e + 1]), minus), l2);
                t = __fadd2_rn(t, make_float2(ex2(a.x), ex2(a.y)));
            }
            s += t.x + t.y;
            return mx;
        };
        const int step = parts * 32;
        // the first element of granule g (whose number modulo 32 is the lane's)
        auto first = [&](int g) { return ALIGNED ? g * GE : (g - lane) * GE + lane; };
        if (lane == 0) sm.count[warp] = 0;
        __syncwarp();
        if (!skip) {
            // (every lane runs the same number of steps: the votes below take the whole warp)
            for (int base = part * 32; base < granules; base += U * step) {
                const int g = base + lane;
                uint4 raw[U];
                float mx[U], top = -INFINITY;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    raw[u] = make_uint4(0, 0, 0, 0);
                    if (g + u * step < whole)
                        raw[u] = ALIGNED ? ld_once(reinterpret_cast<const uint4 *>(row) + (g + u * step))
                                         : load_elements<BF16, ES>(row, first(g + u * step), V);
                }
                if (REST && base + 31 + (U - 1) * step >= whole) {
                    // (the last step of the warps that reach the end; one lane of one of them has the rest of the row)
                    bool mine = false;
#pragma unroll
                    for (int u = 0; u < U; ++u) mine = mine || g + u * step == whole;
                    if (mine) {
                        const uint4 rest = load_elements<BF16, 1>(row, whole * GE, V);
#pragma unroll
                        for (int u = 0; u < U; ++u)
                            if (g + u * step == whole) raw[u] = rest;
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    mx[u] = -INFINITY;
                    if (g + u * step < granules) mx[u] = sum_up(raw[u], first(g + u * step));
                    top = fmaxf(top, mx[u]);
                }
                const unsigned long long shared_thr = *reinterpret_cast<volatile unsigned long long *>(&sm.bound[k]);
                if (shared_thr > thr) thr = shared_thr, thr_x = key_value(thr);
                if (!__any_sync(0xffffffffu, top >= thr_x && top > -INFINITY)) continue;
                if (!seeded) {
                    // K lanes have a maximum of at least this
                    uint32_t o = top > -INFINITY ? order_f32(top) : 0, best = 0;
#pragma unroll 1
                    for (int r = 0; r < K; ++r) {
                        best = __reduce_max_sync(0xffffffffu, o);
                        if (lane == __ffs(__ballot_sync(0xffffffffu, o == best)) - 1) o = 0;
                    }
                    if (best) {
                        thr = (static_cast<unsigned long long>(best) << 32) - 1;
                        thr_x = unorder_f32(best);
                    }
                    seeded = true;
                }
                uint32_t todo = 0;      // granules with a candidate in some lane
#pragma unroll
                for (int u = 0; u < U; ++u)
                    todo |= (__any_sync(0xffffffffu, mx[u] >= thr_x && mx[u] > -INFINITY) ? 1u : 0u) << u;
#pragma unroll 1
                for (; todo; todo &= todo - 1) {
                    const int u = __ffs(todo) - 1;
                    float mu = mx[0];
                    uint4 ru = raw[0];
#pragma unroll
                    for (int w = 1; w < U; ++w)
                        if (u == w) mu = mx[w], ru = raw[w];
                    const bool hit = mu >= thr_x && mu > -INFINITY;
                    const uint32_t hits = __ballot_sync(0xffffffffu, hit);
                    if (!hits) continue;
                    float x[GE];
                    widen<BF16>(ru, x);
                    const int i0 = first(g + u * step);
                    if (count + GE * __popc(hits) <= kSelBuf) {
                        // the few lanes with a candidate push on their own
                        if (hit) {
#pragma unroll
                            for (int e = 0; e < GE; ++e)
                                if (x[e] >= thr_x && x[e] > -INFINITY && i0 + e * ES < V) {
                                    const unsigned long long key = make_key(x[e], i0 + e * ES);
                                    if (key > thr) buf[atomicAdd(&sm.count[warp], 1)] = key;
                                }
                        }
                        __syncwarp();
                        count = *reinterpret_cast<volatile int *>(&sm.count[warp]);
                    } else {
                        // one element of every lane at a time, making room when there is none
#pragma unroll 1
                        for (int e = 0; e < GE; ++e) {
                            if (count > kSelBuf - 32) keep_best();
                            float xe = x[0];
#pragma unroll
                            for (int f = 1; f < GE; ++f) xe = e == f ? x[f] : xe;
                            const unsigned long long key = make_key(xe, i0 + e * ES);
                            const bool in = hit && xe > -INFINITY && i0 + e * ES < V && key > thr;
                            const uint32_t who = __ballot_sync(0xffffffffu, in);
                            if (in) buf[count + __popc(who & ((1u << lane) - 1u))] = key;
                            count += __popc(who);
                        }
                        if (lane == 0) sm.count[warp] = count;
                        __syncwarp();
                    }
                }
                if (count >= 2 * K) keep_best();    // a tighter bound for what follows
            }
        }
        keep_best();
        // the part's maximum and sum
        float mw = m;
#pragma unroll
        for (int o = 16; o; o >>= 1) mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, o));
        s *= ex2((m - mw) * kLog2e);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) sm.m[warp] = mw, sm.s[warp] = s;
    }
    cluster_sync_all();
    // phase 2: merge a row's parts (rows over CTAs first, then over warps)
    for (int k = rank + cs * warp; k < K; k += cs * kSelWarps) {
        const int parts = nw / K;
        SelSmem *home = in_cta(&sm, 0);
        // lse from the parts' maxima and sums
        float mx = -3.402823466e38f;
        for (int i = lane; i < parts; i += 32) {
            const int gw = k + i * K;
            mx = fmaxf(mx, in_cta(&sm, gw / kSelWarps)->m[gw % kSelWarps]);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        double sum = 0.0;
        for (int i = lane; i < parts; i += 32) {
            const int gw = k + i * K;
            SelSmem *at = in_cta(&sm, gw / kSelWarps);
            sum += (double)(at->s[gw % kSelWarps] * ex2((at->m[gw % kSelWarps] - mx) * kLog2e));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) home->row_max[k] = mx, home->row_log[k] = log(sum);
        // the parts' keys, at most 16 CS of them, and K rounds of taking the largest
        constexpr int N = kSelWarps * 8 / 32;
        unsigned long long kp[N];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int i = lane + 32 * u, gw = k + i / K * K;
            kp[u] = i < parts * K ? in_cta(&sm, gw / kSelWarps)->keys[gw % kSelWarps][i % K] : 0;
        }
#pragma unroll 1
        for (int r = 0; r < K; ++r) {
            unsigned long long best = kp[0];
#pragma unroll
            for (int u = 1; u < N; ++u) best = kp[u] > best ? kp[u] : best;
            best = warp_max(best);
            if (lane == r) home->row_keys[k][r] = best;
#pragma unroll
            for (int u = 0; u < N; ++u)
                if (kp[u] == best) kp[u] = 0;
        }
    }
    cluster_sync_all();
    if (rank != 0 || warp != 0) return;
    // phase 3: lane k holds the head of row k; K rounds of taking the best score
    const int k = lane;
    const double score = score_f;
    const double mx = k < K ? sm.row_max[k] : 0.0, lg = k < K ? sm.row_log[k] : 0.0;
    const bool usable = k < K && isfinite(score) && (ended || (isfinite(mx) && isfinite(lg)));
    int pos = 0;
    double cand = 0.0;
    int token = 0;
    unsigned long long ord = 0;   // 0: no candidate left
    auto load_head = [&]() {
        ord = 0;
        if (!usable || pos >= K) return;
        if (ended) {
            if (pos == 0) cand = score, token = args.eos, ord = order_f64(cand);
            return;
        }
        const unsigned long long key = sm.row_keys[k][pos];
        if (!key) return;
        cand = score + (((double)key_value(key) - mx) - lg);
        token = key_index(key);
        ord = order_f64(cand);
    };
    load_head();
    float my_next = -INFINITY;
    int my_parent = lane, my_token = 0;
    bool my_end = ended;
    for (int r = 0; r < K; ++r) {
        const unsigned long long best = warp_max(ord);
        if (!best) break;
        const int win = __ffs(__ballot_sync(0xffffffffu, ord == best)) - 1;   // equal scores: the lower row
        const double c = __shfl_sync(0xffffffffu, cand, win);
        const int tk = __shfl_sync(0xffffffffu, token, win);
        const bool was = __shfl_sync(0xffffffffu, ended ? 1 : 0, win) != 0;
        if (lane == r) my_next = (float)c, my_parent = win, my_token = tk, my_end = was || tk == args.eos;
        if (lane == win) ++pos, load_head();
    }
    // every lane has read its scores and flags: the outputs may lie over them
    __syncwarp();
    if (lane < K) {
        args.next_scores[bk + lane] = my_next;
        args.parents[bk + lane] = my_parent;
        args.tokens[bk + lane] = my_token;
        if (args.done_out) args.done_out[bk + lane] = my_end ? 1 : 0;
    }
}

// ------------------------------------------------------------ state reorder
// Slot j of a request becomes its slot parents[j].  A thread takes one word of
// the slots: it loads that word of every parent of a slot that changes and then stores
// them, so the move may be in place (no thread touches another's word) and a
// parent that several slots share is read from HBM once.  A slot that keeps its
// state is neither read (for itself) nor written when the move is in place.  Bound by
// HBM: 256 states of 1 MB in 64 requests of 4, random parents, take 55 us (359 MB, 97 %
// of the copy bandwidth).
template <typename W, int KM>
__global__ void __launch_bounds__(256)
state_reorder_kernel(const W *S, const W *z, const int *__restrict__ parents, int K, long long s_len,
                     long long z_len, unsigned s_blocks, W *S_out, W *z_out, int *status)
{
    const int b = blockIdx.y;
    const bool norm = blockIdx.x >= s_blocks;
    const W *src = norm ? z : S;
    W *dst = norm ? z_out : S_out;
    const long long len = norm ? z_len : s_len;
    const long long e = (long long)(blockIdx.x - (norm ? s_blocks : 0)) * blockDim.x + threadIdx.x;
    const int *par = parents + (size_t)b * K;
    if (blockIdx.x == 0 && threadIdx.x < K && static_cast<unsigned>(par[threadIdx.x]) >= static_cast<unsigned>(K))
        atomicExch(status, kStatusShape);
    if (e >= len) return;
    const size_t base = (size_t)b * K * len + e;
    const bool in_place = src == dst;
    W v[KM];
    uint32_t moved = 0;
#pragma unroll
    for (int j = 0; j < KM; ++j) {
        if (j >= K) continue;
        const int p = par[j];
        if (static_cast<unsigned>(p) >= static_cast<unsigned>(K) || (in_place && p == j)) continue;
        v[j] = src[base + (size_t)p * len];
        moved |= 1u << j;
    }
#pragma unroll
    for (int j = 0; j < KM; ++j)
        if (moved >> j & 1) dst[base + (size_t)j * len] = v[j];
}

template <typename W>
cudaError_t launch_reorder(const W *S, const W *z, const int *parents, int B, int K, long long s_len, long long z_len,
                           W *S_out, W *z_out, int *status, cudaStream_t stream)
{
    const long long sb = (s_len + 255) / 256, zb = z ? (z_len + 255) / 256 : 0;
    const dim3 grid((unsigned)(sb + zb), B);
    auto run = [&](auto kern) {
        kern<<<grid, 256, 0, stream>>>(S, z, parents, K, s_len, z_len, (unsigned)sb, S_out, z_out, status);
    };
    if (K <= 4) run(state_reorder_kernel<W, 4>);
    else if (K <= 8) run(state_reorder_kernel<W, 8>);
    else if (K <= 16) run(state_reorder_kernel<W, 16>);
    else run(state_reorder_kernel<W, 32>);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_beam_select(const BeamSelectArgs &a, int B, bool bf16, int sms, cudaStream_t stream)
{
    // CTAs per request: as many as keep the batch resident at 2 per SM.  A cluster lies in one GPC and leaves some of
    // its SMs over, so 7/8 of them are counted on: K4 V131072 BF16 at B = 76 takes 48.9 us with 4 (304 CTAs, a second
    // wave) and 37.6 with 3, B = 48 32.2 with 4, 29.6 with 5 and 41.0 with 6, B = 88 46.1 with 2 and 38.1 with 3.
    int cs = 8;
    while (cs > 2 && 4LL * B * cs > 7LL * sms) --cs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cs, B, 1);
    cfg.blockDim = dim3(kSelThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int el = bf16 ? 2 : 4;
    const bool aligned = (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 && a.row_stride * el % 16 == 0;
    auto run = [&](auto kern) { return cudaLaunchKernelEx(&cfg, kern, a); };
    const int ge = 16 / el;
    const bool rest = whole_granules(a.V, ge) * ge < a.V;
    if (bf16)
        return !aligned ? run(beam_select_kernel<true, false, false>)
               : rest   ? run(beam_select_kernel<true, true, true>)
                        : run(beam_select_kernel<true, true, false>);
    return !aligned ? run(beam_select_kernel<false, false, false>)
           : rest   ? run(beam_select_kernel<false, true, true>)
                    : run(beam_select_kernel<false, true, false>);
}

cudaError_t launch_state_reorder(const float *S, const float *z, const int *parents, int B, int K, long long s_len,
                                 long long z_len, float *S_out, float *z_out, int *status, cudaStream_t stream)
{
    auto ok = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    if (s_len % 4 == 0 && ok(S) && ok(S_out) && (!z || (z_len % 4 == 0 && ok(z) && ok(z_out))))
        return launch_reorder(reinterpret_cast<const float4 *>(S), reinterpret_cast<const float4 *>(z), parents, B, K,
                              s_len / 4, z_len / 4, reinterpret_cast<float4 *>(S_out), reinterpret_cast<float4 *>(z_out),
                              status, stream);
    return launch_reorder(S, z, parents, B, K, s_len, z_len, S_out, z_out, status, stream);
}

}  // namespace la
