// dd.cuh -- double-word arithmetic: a value as the unevaluated sum of two
// floats (about 48 bits).  Sums and products are the error-free
// transformations of Dekker and Knuth; the exponential is argument reduction
// by ln 2, a Taylor series and repeated squaring.  On this GPU fp64 runs at
// two lanes a cycle; a score in double words costs about 100 fp32 instructions.
#pragma once
#include <cuda_runtime.h>

#include <cmath>

#include "common.cuh"

namespace kosmos {

struct dd {
    float hi, lo;
};

// A product that is not contracted into a following sum.
KOS_HD float mul_rn(float a, float b) {
#ifdef __CUDA_ARCH__
    return __fmul_rn(a, b);
#else
    volatile float p = a * b;
    return p;
#endif
}

// a + b exactly (|a| >= |b|)
KOS_HD dd quick_two_sum(float a, float b) {
    const float s = a + b;
    return {s, b - (s - a)};
}
// a + b exactly
KOS_HD dd two_sum(float a, float b) {
    const float s = a + b, bb = s - a;
    return {s, (a - (s - bb)) + (b - bb)};
}
KOS_HD dd dd_add(dd a, float b) {
    const dd s = two_sum(a.hi, b);
    return quick_two_sum(s.hi, s.lo + a.lo);
}
KOS_HD dd dd_add(dd a, dd b) {
    const dd s = two_sum(a.hi, b.hi);
    return quick_two_sum(s.hi, s.lo + (a.lo + b.lo));
}
KOS_HD dd dd_mul(dd a, dd b) {
    const float p = mul_rn(a.hi, b.hi);
    float e = fmaf(a.hi, b.hi, -p);
    e = fmaf(a.hi, b.lo, e);
    e = fmaf(a.lo, b.hi, e);
    return quick_two_sum(p, e);
}
// 1 / d for a positive d in fp32's middle range: one Newton step on the fp32 quotient
KOS_HD dd dd_inverse(dd d) {
    const float q = 1.0f / d.hi;
    float r = fmaf(-d.hi, q, 1.0f);
    r = fmaf(-d.lo, q, r);
    return quick_two_sum(q, mul_rn(q, fmaf(r, r, r)));
}

// e^y for y <= 0, off by at most 1e-11 of it (1e-35 absolutely where the low
// word underflows, below e^-60).
// y = n ln 2 + r, e^r = (1 + E)^16 with E = e^(r / 16) - 1.
KOS_HD dd dd_exp(dd y) {
    constexpr float LOG2E_F = 1.4426950408889634f;
    // ln 2 in three parts: 16 bits (a multiple of it by n is exact), 24 bits, the rest
    constexpr float LN2_1 = 45426.0f / 65536.0f, LN2_2 = 0x1.7f7d1cp-20f, LN2_3 = 5.497923e-14f;
    float n = rintf(mul_rn(y.hi, LOG2E_F));
    const bool zero = !(n >= -120.0f);  // no branch: several exponentials run side by side
    if (zero) n = y.hi = y.lo = 0.0f;
    const float r1 = fmaf(-n, LN2_1, y.hi);
    const float p = mul_rn(n, LN2_2);
    dd r = two_sum(r1, -p);
    r = quick_two_sum(r.hi, r.lo + (y.lo - fmaf(n, LN2_2, -p) - mul_rn(n, LN2_3)));
    r = {r.hi * 0.0625f, r.lo * 0.0625f};
    const dd q = dd_mul(r, r);
    // the terms from r^3 / 6 on are under 2e-6: fp32
    const float t = fmaf(r.hi, fmaf(r.hi, fmaf(r.hi, 1.0f / 720.0f, 1.0f / 120.0f), 1.0f / 24.0f), 1.0f / 6.0f);
    const float c = mul_rn(mul_rn(q.hi, r.hi), t);
    dd e = two_sum(r.hi, 0.5f * q.hi);
    e = quick_two_sum(e.hi, e.lo + (r.lo + fmaf(0.5f, q.lo, c)));
    for (int i = 0; i < 4; ++i) {  // (1 + E)^2 - 1 = 2 E + E^2
        const dd sq = dd_mul(e, e);
        e = dd_add({2.0f * e.hi, 2.0f * e.lo}, sq);
    }
    e = dd_add(e, 1.0f);
#ifdef __CUDA_ARCH__
    const float scale = __int_as_float((static_cast<int>(n) + 127) << 23);
#else
    const float scale = ldexpf(1.0f, static_cast<int>(n));
#endif
    return {zero ? 0.0f : e.hi * scale, zero ? 0.0f : e.lo * scale};
}

// 1 / (1 + e^-x), off by at most 2e-11.
KOS_HD dd dd_sigmoid(float x) {
    const dd e = dd_exp({-fabsf(x), 0.0f});
    const dd q = dd_inverse(dd_add(e, 1.0f));
    return x >= 0.0f ? q : dd_mul(e, q);
}

}  // namespace kosmos
