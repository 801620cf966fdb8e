// gdelta_tc.cuh -- what the gated delta rule's tensor-core kernels share: the chunks' workspace, operand splits, TMEM and
// shared-memory accesses.
#pragma once

#include "gdelta_tc.h"
#include "launch_after.cuh"
#include "tc_common.cuh"
#include "tc_short.cuh"

#include <cstddef>

namespace la {
namespace {

constexpr uint32_t kHi128 = desc_hi(1024, 2);   // SBO and swizzle of 128-byte rows
constexpr uint32_t kTile = kC * 128;            // 8 KB: 64 rows of 64 BF16
// workspace per chunk and head: A, X's high and low parts (BF16 shared-memory images), then 64 floats each of e^G, e^{G_C - G}
// and beta.  For the gradients also A's low part and scale e^G Q (two parts of up to two blocks of 64 features), and behind the gates
// log2 e^G as pairs of a high and a low FP32 part (no gate below kLeastGate), the true beta over the one used, and how many gates up to
// the token are below kLeastGate.
constexpr uint32_t kWsA = 0, kWsX = kTile, kWsGates = 3 * kTile, kWsChunk = kWsGates + 1024;
constexpr uint32_t kWsAl = kWsGates + 2048, kWsQ = kWsAl + kTile, kWsChunkB = kWsQ + 4 * kTile;
constexpr uint32_t kGateBytes = 3 * kC * 4, kGateBytesB = 7 * kC * 4;
constexpr uint32_t kGateLog = 3 * kC * 4, kGateRatio = 5 * kC * 4, kGateClosed = 6 * kC * 4;

__device__ __forceinline__ uint8_t *align1024(uint8_t *p)
{
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

__device__ __forceinline__ uint4 pack8(const float *f)
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// 2^x, relative error about 2^-22; 0 below 2^-126
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The sequence and the chunks of a CTA.
struct Span {
    int T;            // tokens of the sequence
    size_t tok0;      // packed: its first token
    size_t slot;      // its first chunk in the workspace (times H heads)
    bool valid;
};

// Packed sequences: slot_base[b] numbers the chunks of all sequences in order; -1 for one whose bounds are invalid.
__device__ __forceinline__ Span span_of(const GdeltaTcArgs &a, int b)
{
    Span s;
    if (!a.s.cu_seqlens) {
        s.T = a.s.T, s.tok0 = 0, s.valid = true;
        s.slot = (size_t)b * ((a.s.T + kC - 1) / kC);
        return s;
    }
    const int base = a.slot_base[b];
    s.valid = base >= 0;
    s.tok0 = s.valid ? a.s.cu_seqlens[b] : 0;
    s.T = s.valid ? a.s.cu_seqlens[b + 1] - (int)s.tok0 : 0;
    s.slot = s.valid ? base : 0;
    return s;
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts_u16(uint32_t a, uint32_t x)
{
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"((uint16_t)x) : "memory");
}
// 8 columns of 32 lanes
__device__ __forceinline__ void tm_ld8(uint32_t a, float (&v)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(a));
}
__device__ __forceinline__ void tm_st8(uint32_t a, const uint32_t (&w)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"r"(a), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
// x as a high and a low BF16 part; the remainders by multiply-adds that take the BF16 parts as they are (5.4 cycles an SM quarter
// per pair and warp, 7.8 with the parts widened first)
__device__ __forceinline__ void split(float2 x, uint32_t &hi, uint32_t &lo)
{
    hi = pack_bf16x2(x.x, x.y);
    float r0, r1;
    asm("{\n\t.reg .b16 a, b, m;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "mov.b16 m, 0xBF80;\n\t"             // -1
        "fma.rn.f32.bf16 %0, a, m, %3;\n\t"
        "fma.rn.f32.bf16 %1, b, m, %4;\n\t}"
        : "=f"(r0), "=f"(r1)
        : "r"(hi), "f"(x.x), "f"(x.y));
    lo = pack_bf16x2(r0, r1);
}
__device__ __forceinline__ float4 lds_f4(uint32_t a)
{
    const uint4 v = lds4(a);
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
// One lane of a converged warp, in a form that keeps what it guards warp-uniform (an MMA's operands then stay in uniform
// registers: 20 cycles to issue one, 45 behind a test of the lane).
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// A warp's way from a column per lane to rows in memory: lane d has 64 tokens of column d, as 32 words of two BF16, and the rows of
// the output have 32 columns (64 bytes) of the warp.  The words go to 128-byte rows of shared memory (4 KB per warp), 16-byte
// word w of row d at w ^ cols_swizzle(d); ldmatrix reads them back transposed, with the rows of its four 8 x 8 matrices chosen so
// that a lane receives eight neighbouring columns of one token.  Neither side has a bank conflict.
__device__ __forceinline__ uint32_t cols_swizzle(int d) { return (d & 1) | ((((d >> 3) ^ (d >> 1)) & 3) << 1); }
// Words 4 w .. 4 w + 3 of this lane's column.
__device__ __forceinline__ void cols_put(uint32_t buf, int lane, int w, uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3)
{
    sts4(buf + lane * 128 + ((w ^ cols_swizzle(lane)) << 4), x0, x1, x2, x3);
}
// Tokens 8 w .. 8 w + 7: this lane gets columns 8 (lane % 4) .. of token 8 w + lane / 4.
__device__ __forceinline__ uint4 cols_get(uint32_t buf, int lane, int w)
{
    const int i = lane & 7, d = 8 * (i >> 1) + 2 * (lane >> 3) + (i & 1);
    uint4 v;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(buf + d * 128 + ((w ^ cols_swizzle(d)) << 4))
                 : "memory");
    return v;
}

// 16 BF16 values (8 words) of one row of a tile in memory with 128-byte rows and the 128-byte swizzle: 16-byte words 2 x and
// 2 x + 1 of the row, which the swizzle leaves side by side (exchanged in odd rows): one 32-byte store.
__device__ __forceinline__ void st_row16(uint8_t *tile, int row, int x, const uint32_t (&w)[8])
{
    const bool odd = row & 1;
    uint8_t *p = tile + row * 128 + ((x ^ ((row & 7) >> 1)) << 5);
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"l"(p), "r"(odd ? w[4] : w[0]), "r"(odd ? w[5] : w[1]), "r"(odd ? w[6] : w[2]), "r"(odd ? w[7] : w[3]),
                   "r"(odd ? w[0] : w[4]), "r"(odd ? w[1] : w[5]), "r"(odd ? w[2] : w[6]), "r"(odd ? w[3] : w[7])
                 : "memory");
}

__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

}  // namespace
}  // namespace la
