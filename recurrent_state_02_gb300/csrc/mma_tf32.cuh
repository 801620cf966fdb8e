// mma_tf32.cuh -- warp-wide products of FP32 numbers in two TF32 parts, for tiles too small for the CTA-wide tensor core.
#pragma once

#include <cstdint>

namespace la {
namespace {

// c += A B, A 16 x 8, B 8 x 8: with g = lane / 4 and t = lane % 4, a = A(g, t), (g + 8, t), (g, t + 4), (g + 8, t + 4), b = B(t, g), (t + 4, g),
// c = C(g, 2 t), (g, 2 t + 1), (g + 8, 2 t), (g + 8, 2 t + 1)
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x as two TF32 numbers, 11 bits of it and the next 11, cut off: less than 2^-20 of it is lost
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo)
{
    hi = __float_as_uint(x) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
}

// The same with the first one rounded to nearest, so that the second one has either sign and what is lost (less than 2^-21) no bias: sums of
// many terms are then as good as in FP32 (cut off, all terms shrink alike)
__device__ __forceinline__ void split_tf32_near(float x, uint32_t &hi, uint32_t &lo)
{
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
}

}  // namespace
}  // namespace la
