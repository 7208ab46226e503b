// Scalar helpers on the FMA pipe, for kernels whose MUFU unit is busy with the softmax
// exponentials: a reciprocal and a base-2 exponential. Both are this library's own
// (a numerically fitted seed with Newton steps; a fitted polynomial), checked on the
// GPU against float64 references by hils_selftest_fast_math.
#pragma once
#include <cuda_runtime.h>

namespace hils {

// 1/z for a normal positive z on the FMA pipe: an integer-subtraction seed (relative
// error at most 5.1e-2, constant fitted numerically over one binade) and two Newton
// steps r <- r (2 - z r), which square the error: below 7e-6 plus rounding.
__device__ __forceinline__ float recip_newton(float z) {
    float r = __int_as_float(0x7ef311c2 - __float_as_int(z));
    r = fmaf(r, fmaf(-z, r, 1.f), r);
    r = fmaf(r, fmaf(-z, r, 1.f), r);
    return r;
}

// 2^x on the FMA pipe (no MUFU), for finite x: x = j + f with j = round(x) (the
// 1.5 * 2^23 shifter) and f in [-1/2, 1/2]; 2^f by a degree-5 polynomial fitted here for
// relative error (iteratively reweighted least squares on Chebyshev nodes; at most
// 2.4e-7 in float32 Horner form); 2^j added to the exponent field. x is clamped to
// [-125, 127] so the result stays a normal float (2^-125 stands for anything smaller).
__device__ __forceinline__ float exp2_fma(float x) {
    x = fminf(fmaxf(x, -125.f), 127.f);
    const float t = x + 12582912.f;
    const float f = x - (t - 12582912.f);
    float p = 1.327647129e-03f;
    p = fmaf(p, f, 9.675540961e-03f);
    p = fmaf(p, f, 5.550713092e-02f);
    p = fmaf(p, f, 2.402212024e-01f);
    p = fmaf(p, f, 6.931469440e-01f);
    p = fmaf(p, f, 1.000000119e+00f);
    return __int_as_float(__float_as_int(p) + ((__float_as_int(t) - 0x4b400000) << 23));
}

// The same for two values that are at most 127, in packed float32 arithmetic: 13 instructions
// for the pair. Below -126 the result is some subnormal number, below -127 (-inf too) 2^-149.
__device__ __forceinline__ float2 exp2_fma2(float2 x) {
    auto fma = [](float2 a, float2 b, float2 c) {
        float2 d;
        asm("fma.rn.f32x2 %0, %1, %2, %3;"
            : "=l"(reinterpret_cast<unsigned long long &>(d))
            : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)),
              "l"(reinterpret_cast<unsigned long long &>(c)));
        return d;
    };
    auto add = [](float2 a, float2 b) {
        float2 d;
        asm("add.rn.f32x2 %0, %1, %2;"
            : "=l"(reinterpret_cast<unsigned long long &>(d))
            : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)));
        return d;
    };
    auto both = [](float c) { return make_float2(c, c); };
    x = make_float2(fmaxf(x.x, -127.f), fmaxf(x.y, -127.f));
    const float2 t = add(x, both(12582912.f));
    const float2 f = fma(add(t, both(-12582912.f)), both(-1.f), x);
    float2 p = fma(both(1.327647129e-03f), f, both(9.675540961e-03f));
    p = fma(p, f, both(5.550713092e-02f));
    p = fma(p, f, both(2.402212024e-01f));
    p = fma(p, f, both(6.931469440e-01f));
    p = fma(p, f, both(1.000000119e+00f));
    // t holds 0x4b400000 + j: shifted left by 23 its upper bits fall away
    return make_float2(__int_as_float(__float_as_int(p.x) + (__float_as_int(t.x) << 23)),
                       __int_as_float(__float_as_int(p.y) + (__float_as_int(t.y) << 23)));
}

}  // namespace hils
