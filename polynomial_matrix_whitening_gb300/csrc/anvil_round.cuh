// anvil_round.cuh -- correctly rounded fp32 quotients and square roots of packed pairs, without the
// branches of the general ones, for operands in the middle of the range.
//
// Both start from the hardware's approximation, refine it by Newton's iteration and end with
// Markstein's correction (P. W. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM J. Res. Dev. 34, 1990): from a quotient q within an ulp and the correctly
// rounded reciprocal y of b, q + (a - b q) y rounds to a / b, since the remainder a - b q is exact in
// one fused operation; the square root's correction is g + (v - g g) h with h near 1 / (2 sqrt v).
// tests/test_gpu_adamw_rounding.py compares AdamW's steps, which are these operations, with the correctly rounded
// ones: the root of every significand at either parity of the exponent (scaling by powers of four changes
// nothing else), and with it every significand of the divisor; 2^26 quotients, a fourth of them as near to the
// middle between two values as any.
#pragma once

#include <stdint.h>

#include "anvil_device.cuh"
#include "anvil_types.cuh"

namespace anvil {

__device__ __forceinline__ float approx_rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float approx_rsqrt(float v) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// (a.x / b.x, a.y / b.y) for b within 2^-60 to 2^90 and |a| within 2^-102 to 2^60 with a quotient from 2^-126 on,
// or a = 0.  (Elsewhere the remainder is not exact, and the quotient off by two ulps at most.)
__device__ __forceinline__ uint64_t f2_divide(uint64_t a, uint64_t b) {
    const uint64_t one = f2_make(1.f, 1.f), nb = f2_neg(b);
    float b0, b1;
    f2_split(b, &b0, &b1);
    uint64_t y = f2_make(approx_rcp(b0), approx_rcp(b1));
    y = f2_fma(f2_fma(nb, y, one), y, y);
    uint64_t q = f2_mul(a, y);
    q = f2_fma(f2_fma(nb, q, a), y, q);
    return f2_fma(f2_fma(nb, q, a), y, q);
}

// (sqrt v.x, sqrt v.y) for v from the smallest value to 2^26, or 0: of 2^100 v, which is exact and in the
// middle of the range.
__device__ __forceinline__ uint64_t f2_root(uint64_t v) {
    v = f2_mul(v, f2_make(0x1p100f, 0x1p100f));
    float v0, v1;
    f2_split(v, &v0, &v1);
    const float least = 0x1p-60f;  // of 0 the approximation is infinite: 0 times this one's is 0
    const uint64_t half = f2_make(0.5f, 0.5f);
    const uint64_t y = f2_make(approx_rsqrt(fmaxf(v0, least)), approx_rsqrt(fmaxf(v1, least)));
    uint64_t g = f2_mul(v, y), h = f2_mul(y, half);
    const uint64_t r = f2_fma(f2_neg(g), h, half);
    g = f2_fma(g, r, g);
    h = f2_fma(h, r, h);
    return f2_mul(f2_fma(f2_fma(f2_neg(g), g, v), h, g), f2_make(0x1p-50f, 0x1p-50f));
}

}  // namespace anvil
