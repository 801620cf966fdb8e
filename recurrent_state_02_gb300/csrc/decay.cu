// decay.cu -- linear attention with a constant decay per head on CUDA cores: the
// token recurrence (any sizes, FP32 arithmetic) and the single-token decode step.
//
//     S_t = g S_{t-1} + k_t v_t^T,   y_t = scale q_t^T S_t
//
// There is no feature map and no normaliser; g is a constant of the head.

#include "decay.h"
#include "launch_rules.h"
#include "sm103_ptx.cuh"

#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

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

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address in CTA `rank` of the cluster of what is at shared address `addr` here.
__device__ __forceinline__ uint32_t in_cluster(uint32_t addr, uint32_t rank)
{
    uint32_t out;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(out) : "r"(addr), "r"(rank));
    return out;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr)
{
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr));
    return x;
}

// ------------------------------------------------------- token recurrence
// One CTA per (b, h, 32 columns), the state in registers.  Its W * CB warps (CB = 4 / CPL) split
// the rows into blocks of 32 and the columns into blocks of 8 CPL; lane (g, jj), g = lane / 8,
// holds rows 8 g .. 8 g + 7 of its warp's in CPL columns.  A token costs a warp four 16-byte
// shared loads of its rows' q and k, one of its columns' v, 12 CPL packed FP32 instructions (row
// pairs: k v, g S + k v, the sum with q) and one store of its partial sums; the 4 W partial outputs of a
// column are added once per block of TB tokens.
// The columns per lane set how a token's time divides.  Loads that a whole warp shares still take shared
// memory about two cycles each, so few columns per lane load it; many make a token's chain of instructions
// long.  One CTA per SM at most (us, FP32, T = 1001): r = 64 82 with CPL = 1, 104 with 2, 203 with 4; r = 128 156, 129,
// 157.  More CTAs, up to 64 rows: 2 (4 in brackets), us: 512 of r = 64 (T = 1000) 239 (277), 4096 of r = 64 and 16 tokens
// 37 (41), 48 packed FP32 prompts of 128 .. 2048 tokens (H = 16, r = dv = 64) 575 (760), 1000 packed BF16 requests of
// 12 tokens 402 (463); only 1024 CTAs of r = 32 lose, 22 (20) at 64 tokens.  More rows: 256 CTAs of r = 128 (T = 1000) 233
// (249), but brief ones, where the state's traffic counts, take 4: 4096 of r = 128 and 8 tokens (BF16) 54 (45), the 48
// prompts at r = dv = 128 1620 (1406), 1000 requests of 12 tokens at r = 256 2380 (1647); one prompt of 2048 tokens among
// 255 of 8 at r = 128 loses, 348 (383).
// Tokens are staged in blocks; the next block's values are fetched into registers while this
// one is computed.
//
// SPLIT: few CTAs leave SMs idle while each walks its tokens one by one, 80 to 230 ns each.  A cluster then takes
// one (b, h, 32 columns), a CTA a segment of its tokens: all form what their segment adds to the state
// from zero (the first one from S_init, with its outputs), exchange the sums over distributed shared
// memory, S <- g^seg S + sum over the segments before, and pass their tokens again with outputs.
constexpr int kRecCols = 32, kRecRows = 32;
constexpr int kRecShort = 64;         // tokens

template <int W, int CPL>
struct RecCfg {
    static constexpr int R = W * kRecRows, CB = 4 / CPL, NW = W * CB, kThreads = 32 * NW;
    static constexpr int TB = W <= 2 ? 32 : W == 4 ? 16 : 8;    // tokens per staged block
    static constexpr int NA = TB / CB;                          // staged a (or b) values per thread
    static constexpr int NC = (TB + NW - 1) / NW;
    static constexpr uint32_t kSmem = 4 * (2 * TB * R + TB * kRecCols + 4 * W * TB * kRecCols);
};

struct RecArgs {
    DecaySweep sw[3];
    DecayArgs d;
    int tiles[3];   // column tiles of each sweep
    int nseg, seg;  // segments of a sequence, one CTA of a cluster each, and their tokens
};

__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 lo2(float4 a) { return make_float2(a.x, a.y); }
__device__ __forceinline__ float2 hi2(float4 a) { return make_float2(a.z, a.w); }

template <bool BF16, int W, int CPL, bool SPLIT>
__global__ void __launch_bounds__(32 * W * 4 / CPL)
decay_rec_kernel(const __grid_constant__ RecArgs args)
{
    using C = RecCfg<W, CPL>;
    constexpr int R = C::R, TB = C::TB, NT = C::kThreads, NW = C::NW;
    extern __shared__ float4 rec_smem[];
    float *as = reinterpret_cast<float *>(rec_smem), *bs = as + TB * R, *cs = bs + TB * R;
    float *ys = cs + TB * kRecCols;              // [4 W][TB][kRecCols]
    const int rank = SPLIT ? blockIdx.x % args.nseg : 0;   // (the cluster spans nseg CTAs of the x axis)
    int tile = SPLIT ? blockIdx.x / args.nseg : blockIdx.x, which = 0;
    while (tile >= args.tiles[which]) tile -= args.tiles[which++];
    const DecaySweep &sw = args.sw[which];
    const DecayArgs &d = args.d;
    const int h = blockIdx.y, b = blockIdx.z, H = d.H, ra = sw.ra, n = sw.n;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
    // the sweep's token t is row first + t * step of a, b (rows of ra elements) and c, out (of n)
    const long long step = (sw.rev ? -1 : 1) * (packed ? (long long)H : 1);
    const long long first = (packed ? (long long)seq0 * H + h : (long long)bh * T) + (sw.rev ? -step * (T - 1) : 0);
    const float g = d.decay[h];
    const int c0 = tile * kRecCols, wr = warp % W, part = lane >> 3;
    const int j1 = (warp / W * 8 + (lane & 7)) * CPL, j0 = c0 + j1;   // this lane's first column
    const int i0 = wr * kRecRows + part * 8;                          // its 8 rows, as 4 pairs

    float2 s[4][CPL];     // [row pair][column]
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            const int i = i0 + 2 * p, j = j0 + c;
            // element i of column j: rows apart, or contiguous in a transposed state
            const float *src = sw.S_init + (sw.init_t ? (bh * n + j) * ra : bh * ra * n + j);
            const size_t step = sw.init_t ? 1 : n;
            const bool ok = sw.S_init && j < n && rank == 0;
            s[p][c] = make_float2(ok && i < ra ? src[i * step] : 0.f, ok && i + 1 < ra ? src[(i + 1) * step] : 0.f);
        }
    // staging: thread e + R x fetches element e of the tokens x, x + CB, .. of a and b; warp w column
    // `lane` of the tokens w, w + NW, .. of c
    float pa[C::NA], pb[C::NA], pc[C::NC];
    const int ea = tid % R, xa = tid / R;
    const bool in_a = ea < ra, in_c = c0 + lane < n;
    const long long sa = step * ra, sc = step * n;
    // the tokens begin .. end-1; `outs`: with their outputs (else the state alone)
    auto pass = [&](int begin, int end, auto outs) {
        constexpr bool OUT = decltype(outs)::value;
        // this thread's first elements at token t0
        long long oa = (first + (begin + xa) * step) * ra + ea, oc = (first + (begin + warp) * step) * n + c0 + lane;
        auto fetch = [&](int t0) {
#pragma unroll
            for (int x = 0; x < C::NA; ++x) {
                const bool ok = in_a && t0 + x * C::CB + xa < end;
                if (OUT) pa[x] = ok ? load_elem<BF16>(sw.a, oa + x * C::CB * sa) : 0.f;
                pb[x] = ok ? load_elem<BF16>(sw.b, oa + x * C::CB * sa) : 0.f;
            }
#pragma unroll
            for (int x = 0; x < C::NC; ++x) {
                const int t = x * NW + warp;
                pc[x] = in_c && t < TB && t0 + t < end ? load_elem<BF16>(sw.c, oc + x * NW * sc) * sw.write_scale : 0.f;
            }
            oa += TB * sa;
        };
        if (begin < end) fetch(begin);
        for (int t0 = begin; t0 < end; t0 += TB) {
            const int nt = min(TB, end - t0);
#pragma unroll
            for (int x = 0; x < C::NA; ++x) {
                if (OUT) as[x * NT + tid] = pa[x];
                bs[x * NT + tid] = pb[x];
            }
#pragma unroll
            for (int x = 0; x < C::NC; ++x)
                if (NW * C::NC == TB || x * NW + warp < TB) cs[x * NT + tid] = pc[x];
            __syncthreads();
            const long long oy = oc;    // of the outputs too
            oc += TB * sc;
            if (t0 + TB < end) fetch(t0 + TB);
            // a token's operands are loaded while the token before is computed
            struct Token {
                float4 x0, x1, k0, k1;
                float v[CPL];
            };
            auto load_token = [&](int t) {
                const float4 *a4 = reinterpret_cast<const float4 *>(as + t * R + i0), *b4 = reinterpret_cast<const float4 *>(bs + t * R + i0);
                Token k;
                if (OUT) k.x0 = a4[0], k.x1 = a4[1];
                k.k0 = b4[0], k.k1 = b4[1];
                if constexpr (CPL == 4) {
                    const float4 v4 = *reinterpret_cast<const float4 *>(cs + t * kRecCols + j1);
                    k.v[0] = v4.x, k.v[1] = v4.y, k.v[2] = v4.z, k.v[3] = v4.w;
                } else if constexpr (CPL == 1) {
                    k.v[0] = cs[t * kRecCols + j1];
                } else {
                    const float2 v2 = *reinterpret_cast<const float2 *>(cs + t * kRecCols + j1);
                    k.v[0] = v2.x, k.v[1] = v2.y;
                }
                return k;
            };
            Token next = load_token(0);
#pragma unroll 2
            for (int t = 0; t < nt; ++t) {
                const Token now = next;
                next = load_token(t + 1 < nt ? t + 1 : t);
                const float2 f = splat(sw.late && t0 + t == 0 ? 1.f : g);
                float2 x[4];
                if (OUT) x[0] = lo2(now.x0), x[1] = hi2(now.x0), x[2] = lo2(now.x1), x[3] = hi2(now.x1);
                const float2 k[4] = {lo2(now.k0), hi2(now.k0), lo2(now.k1), hi2(now.k1)};
                float2 y[CPL] = {};
#pragma unroll
                for (int p = 0; p < 4; ++p)
#pragma unroll
                    for (int c = 0; c < CPL; ++c) {
                        s[p][c] = __ffma2_rn(f, s[p][c], __fmul2_rn(k[p], splat(now.v[c])));
                        if (OUT) y[c] = __ffma2_rn(x[p], s[p][c], y[c]);
                    }
                if (!OUT) continue;
                float *yt = ys + ((4 * wr + part) * TB + t) * kRecCols + j1;
                if constexpr (CPL == 4)
                    *reinterpret_cast<float4 *>(yt) = make_float4(y[0].x + y[0].y, y[1].x + y[1].y, y[2].x + y[2].y, y[3].x + y[3].y);
                else if constexpr (CPL == 1)
                    *yt = y[0].x + y[0].y;
                else
                    *reinterpret_cast<float2 *>(yt) = make_float2(y[0].x + y[0].y, y[1].x + y[1].y);
            }
            __syncthreads();
            if (!OUT) continue;
#pragma unroll
            for (int x = 0; x < C::NC; ++x) {
                if (x * NW + warp >= nt) break;
                float y = 0.f;
#pragma unroll
                for (int w = 0; w < 4 * W; ++w) y += ys[w * TB * kRecCols + x * NT + tid];
                if (in_c) store_elem<BF16>(sw.out, oy + x * NW * sc, y * sw.out_scale);
            }
            // (the next iteration's first barrier orders these reads of ys before its next writes, and
            // this iteration's last one its reads of the staged tokens before they are overwritten)
        }
    };
    if constexpr (!SPLIT) {
        pass(0, T, std::true_type{});
    } else {
        // what each segment adds to the state (the first one: its final state, and its outputs) ..
        const int begin = rank * args.seg, end = min(T, begin + args.seg);
        const bool last = rank == args.nseg - 1;
        if (rank == 0) pass(begin, end, std::true_type{});
        else if (!last) pass(begin, end, std::false_type{});
        __syncthreads();
        if (!last) {
            // .. to the CTAs behind it, in the words of ys (R x kRecCols of them are there); a thread
            // holds the same elements in every CTA
#pragma unroll
            for (int p = 0; p < 4; ++p)
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    ys[((2 * p) * CPL + c) * NT + tid] = s[p][c].x;
                    ys[((2 * p + 1) * CPL + c) * NT + tid] = s[p][c].y;
                }
        }
        cluster_sync();
        if (rank > 0) {
            // g^seg by repeated squares in 64 bits
            double gp = 1.0, gb = g;
            for (int e = args.seg; e; e >>= 1, gb *= gb)
                if (e & 1) gp *= gb;
            const float gs = static_cast<float>(gp);
            for (int part_rank = 0; part_rank < rank; ++part_rank) {
                const uint32_t from = in_cluster(smem_u32(ys + tid), part_rank);
#pragma unroll
                for (int p = 0; p < 4; ++p)
#pragma unroll
                    for (int c = 0; c < CPL; ++c) {
                        const float x0 = ld_cluster(from + 4 * ((2 * p) * CPL + c) * NT);
                        const float x1 = ld_cluster(from + 4 * ((2 * p + 1) * CPL + c) * NT);
                        s[p][c] = part_rank ? make_float2(fmaf(gs, s[p][c].x, x0), fmaf(gs, s[p][c].y, x1)) : make_float2(x0, x1);
                    }
            }
        }
        cluster_sync();   // (every CTA's ys has been read)
        if (rank > 0) pass(begin, end, std::true_type{});
        if (!last) return;
    }
    if (!sw.S_fin) return;
    const float f = sw.late && T > 0 ? g : 1.f;
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = i0 + 2 * p + e;
            if (i >= ra) continue;
            float *dst = sw.S_fin + bh * ra * n + (size_t)i * n + j0;
#pragma unroll
            for (int c = 0; c < CPL; ++c)
                if (j0 + c < n) dst[c] = (e ? s[p][c].y : s[p][c].x) * f;
        }
}

template <bool BF16, int W, int CPL, bool SPLIT = false>
cudaError_t launch_rec_w(const RecArgs &r, dim3 grid, cudaStream_t stream)
{
    using C = RecCfg<W, CPL>;
    if (!SPLIT) {    // (rec_room has set the attributes of a split instance)
        static OncePerDevice once;
        const cudaError_t e = set_smem_once(decay_rec_kernel<BF16, W, CPL, SPLIT>, C::kSmem, once);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = SPLIT ? dim3(grid.x * r.nseg, grid.y, grid.z) : grid;
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = SPLIT ? r.nseg : 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = SPLIT ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, decay_rec_kernel<BF16, W, CPL, SPLIT>, r);
}

// Clusters of 2 .. kMaxRecSegments CTAs of a split instance that the device places at once with one CTA per SM, and with two.
// Asked of the CUDA driver once per device, as it depends on the GPCs that the device (or a partition of it) has; what the
// CUDA driver cannot answer counts as no room.  (152 SMs: 15 clusters of 8 with an SM per CTA, 8 of 12, 7 of 16.)
struct RecRoom {
    int one[kMaxRecSegments + 1], two[kMaxRecSegments + 1];
};

template <bool BF16, int W, int CPL>
RecRoom rec_room()
{
    static std::atomic<int> one[kMaxDevices][kMaxRecSegments + 1], two[kMaxDevices][kMaxRecSegments + 1];
    static OncePerDevice once;
    RecRoom room = {};
    const int dev = current_device_index();
    if (dev < 0) return room;
    if (!once.done[dev].load(std::memory_order_acquire)) {
        // shared memory that leaves an SM room for one CTA, or for two
        constexpr int kOne = 120 * 1024, kTwo = 80 * 1024;
        static_assert(RecCfg<W, CPL>::kSmem <= kTwo, "an SM holds two CTAs");
        auto kern = decay_rec_kernel<BF16, W, CPL, true>;
        auto works = [](cudaError_t e) {
            if (e != cudaSuccess) cudaGetLastError();    // (an answer of no is not an error of the caller's)
            return e == cudaSuccess;
        };
        if (works(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kOne)) &&
            works(cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1))) {
            for (int n = 2; n <= kMaxRecSegments; ++n) {
                cudaLaunchConfig_t cfg = {};
                cfg.gridDim = dim3(n, 1, 1);
                cfg.blockDim = dim3(RecCfg<W, CPL>::kThreads, 1, 1);
                cudaLaunchAttribute attr[1];
                attr[0].id = cudaLaunchAttributeClusterDimension;
                attr[0].val.clusterDim.x = n;
                attr[0].val.clusterDim.y = 1;
                attr[0].val.clusterDim.z = 1;
                cfg.attrs = attr;
                cfg.numAttrs = 1;
                auto clusters = [&](int smem) {
                    cfg.dynamicSmemBytes = smem;
                    int k = 0;
                    return works(cudaOccupancyMaxActiveClusters(&k, kern, &cfg)) ? k : 0;
                };
                one[dev][n].store(clusters(kOne), std::memory_order_relaxed);
                two[dev][n].store(clusters(kTwo), std::memory_order_relaxed);
            }
        }
        once.done[dev].store(true, std::memory_order_release);
    }
    for (int n = 2; n <= kMaxRecSegments; ++n) {
        room.one[n] = one[dev][n].load(std::memory_order_relaxed);
        room.two[n] = two[dev][n].load(std::memory_order_relaxed);
    }
    return room;
}

template <bool BF16, int W, int FEW, int MANY>
cudaError_t launch_rec_rows(RecArgs r, int rows, dim3 grid, cudaStream_t stream)
{
    const long long ctas = (long long)grid.x * grid.y * grid.z;
    if (!r.d.cu_seqlens && r.d.T >= kMinRecSplit) {
        const RecRoom room = rec_room<BF16, W, FEW>();
        const int want = rec_segments(ctas, rows, r.d.T, room.one, room.two);
        if (want > 1) {
            r.seg = (r.d.T + want - 1) / want;
            r.nseg = (r.d.T + r.seg - 1) / r.seg;
            return launch_rec_w<BF16, W, FEW, true>(r, grid, stream);
        }
    }
    const bool brief = r.d.cu_seqlens || r.d.T <= kRecShort;
    return rec_columns(rows, ctas, brief, r.d.sms) == FEW ? launch_rec_w<BF16, W, FEW>(r, grid, stream)
                                                          : launch_rec_w<BF16, W, MANY>(r, grid, stream);
}

template <bool BF16>
cudaError_t launch_rec(const RecArgs &r, int rows, dim3 grid, cudaStream_t stream)
{
    if (rows <= 32) return launch_rec_rows<BF16, 1, 1, 2>(r, rows, grid, stream);
    if (rows <= 64) return launch_rec_rows<BF16, 2, 1, 2>(r, rows, grid, stream);
    if (rows <= 128) return launch_rec_rows<BF16, 4, 2, 4>(r, rows, grid, stream);
    return launch_rec_rows<BF16, 8, 2, 4>(r, rows, grid, stream);
}

// ------------------------------------------------------------ decode step
// Reads and rewrites r dv FP32 state words per head, two FMAs each: bound by HBM.
// CTA (b, h) of 8 warps; a warp takes RW rows, its lanes 4 columns each, and
// issues every state load before any arithmetic.  B256 H16 r = dv = 128: 81.3 us, 6.6
// TB/s, 99 % of the copy bandwidth; one request's 16 heads: 2.8 us.
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
    r.nseg = 1, r.seg = a.T;
    return bf16 ? launch_rec<true>(r, rows, grid, stream) : launch_rec<false>(r, rows, grid, stream);
}

cudaError_t launch_decay_decode(const void *q, const void *k, const void *v, bool bf16, const float *decay, float *S,
                                int B, int H, int r, int dv, float scale, void *y, cudaStream_t stream)
{
    return bf16 ? launch_dec<true>(q, k, v, decay, S, B * H, H, r, dv, scale, y, stream)
                : launch_dec<false>(q, k, v, decay, S, B * H, H, r, dv, scale, y, stream);
}

}  // namespace la
