// kt_exact.cuh -- fp32 arithmetic on pairs, every operation correctly rounded: what AdamW and the 8-bit floating point
// quantiser have in common.
#pragma once
#include "kt_gemm.cuh"

namespace kt {

// The sum of a product and another number, each rounded: the assembler makes one rounding of a paired product and a paired
// sum, .rn or not, but cannot where the sum is a product with a one that it does not know.
__device__ __forceinline__ f32x2 sum_rn(f32x2 product, f32x2 other, f32x2 one) { return f2_fma<true>(product, one, other); }

// Correctly rounded square roots and quotients of pairs by the method of Markstein (Computation of elementary functions
// on the IBM RISC System/6000 processor, 1990): an approximation, refined once, and a last step from the exact
// residue.  For operands whose intermediate results are normal numbers (the caller's check).  The last step of a quotient
// wants the reciprocal that is nearest to 1 / b.  One refinement gives that from any approximation to one unit, but for 32
// significands of b whose reciprocals lie next to the middle of two numbers: quotients such as 1.0 / 0x1.fffffep+0 and
// 0x1.aaaaa6p+0 / 0x1.fffffap+0 could then be one unit off.  This hardware's approximation is good enough there too: the
// tests try every divisor's and every root's significand.  At a time of two values they take a third of the instructions
// of __fsqrt_rn and __fdiv_rn, whose branches for the other operands are taken per value.
__device__ __forceinline__ float rsqrt_approx(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// (h, and v at the end, are taken with the other sign, as the paired instructions have no sign of their own)
__device__ __forceinline__ f32x2 root_rn(f32x2 v) {
    const f32x2 y = f2(rsqrt_approx(v.x), rsqrt_approx(v.y));
    f32x2 g = f2_mul<true>(v, y), h = f2_mul<true>(y, f2(-0.5f));
    const f32x2 e = f2_fma<true>(h, g, f2(0.5f));
    g = f2_fma<true>(g, e, g);
    h = f2_fma<true>(h, e, h);
    return f2_fma<true>(f2_fma<true>(g, g, f2_mul<true>(v, f2(-1.0f))), h, g);
}
// a / b; nb: -b
__device__ __forceinline__ f32x2 quotient_rn(f32x2 a, f32x2 b, f32x2 nb) {
    f32x2 y = f2_rcp(b);
    y = f2_fma<true>(y, f2_fma<true>(nb, y, f2(1.0f)), y);
    const f32x2 q = f2_mul<true>(a, y);
    return f2_fma<true>(f2_fma<true>(nb, q, a), y, q);
}

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN if either is one
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {  // of those that are no NaN
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

}  // namespace kt
