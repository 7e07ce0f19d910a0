// The soft cap of attention scores, c tanh(s / c), for scores in any unit.
//
// Below half the cap an odd polynomial in x = s / c, whose relative error is 2^-23 (a fit of
// tanh(x) / x in x^2 on [0, 1/4], smallest largest relative error, by exchange: 2^-26 before
// its coefficients are rounded), above it 1 - 2 / (1 + e^2|x|), whose error of 2^-22 is that of
// a value of 0.46 or more.  So the result is within a few 2^-22 of its own size, however
// large the cap; a NaN stays one.
//
// And the slope of a distance bias.  From 2^13 a token on, a token's weight is below e^-8192 of
// its nearer neighbour's: larger slopes count as that.  Below 2^14 in units of log 2, times 2^31
// tokens at most, a bias is far inside float32's range, whatever finite slope is asked for (a
// slope of 3e38 made rows NaN: infinity times a distance of 0, or less another infinity).
#pragma once

#include <stdint.h>

namespace pgd {

__device__ __forceinline__ float tanh_near(float x) {  // |x| < 1/2
    const float z = x * x;
    float p = fmaf(z, 0.017135007f, -0.052986074f);
    p = fmaf(p, z, 0.13324779f);
    p = fmaf(p, z, -0.33333069f);
    return fmaf(p * z, x, x);
}
__device__ __forceinline__ float capped(float s, float cap, float inv) {
    const float x = s * inv, p = tanh_near(x);
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fabsf(x) * 2.8853900817779268f));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    const float big = copysignf(fmaf(-2.f, r, 1.f), x);
    return cap * (fabsf(x) < 0.5f ? p : big);
}

constexpr float kMostSlope = 8192.f;
// In units of log 2 a token, from natural ones.
__device__ __forceinline__ float slope_of(const float* slope) {
    return fminf(fmaxf(__ldg(slope), -kMostSlope), kMostSlope) * 1.4426950408889634f;
}

}  // namespace pgd
