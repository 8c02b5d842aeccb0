// Many binary32 quotients by one divisor, each rounded to nearest even as the division is.
#pragma once

#include "lm_common.cuh"

namespace moedc {

// By Markstein's theorem (Computation of elementary functions on the IBM RISC System/6000
// processor, 1990): with y the correctly rounded 1 / b and q within an ulp of a / b, q + (a -
// q b) y, both in one rounding, is the correctly rounded quotient.  a y is within two ulps;
// one correction brings it within one, the next one is the theorem's.  Where q is so small
// that a - q b leaves binary32 its code is 0 all the same.  Divisors are positive; an infinite
// one divides.
// kSteps 1: only the last correction.  For dividends of up to 11 significant bits (bf16, f16)
// that has been enough for every pair of mantissas (tests/cuda/quotient_sweep.cu).
template <int kSteps> struct Quotient {
    float b, y;
    static __device__ __forceinline__ Quotient by(float divisor)
    {
        Quotient q;
        q.b = divisor;
        q.y = __frcp_rn(divisor);
        return q;
    }
    __device__ __forceinline__ float2 of(float2 a) const
    {
        if (b > 3.4e38f) return make_float2(__fdiv_rn(a.x, b), __fdiv_rn(a.y, b));
        const float2 minus = splat2(-b), by = splat2(y);
        float2 q = mul2_rn(a, by);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) q = fma2_rn(fma2_rn(q, minus, a), by, q);
        // the corrections turn -0 to +0
        return make_float2(copysignf(q.x, a.x), copysignf(q.y, a.y));
    }
    // two e4m3 codes, low byte first
    __device__ __forceinline__ uint32_t codes(float a0, float a1) const
    {
        const float2 q = of(make_float2(a0, a1));
        return pack_e4m3x2(q.x, q.y);
    }
};

}  // namespace moedc
