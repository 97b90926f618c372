// Activations of the gated unit and of the group norm, with their slopes.
#pragma once

#include <hip/hip_runtime.h>

#include "block.hpp"

namespace iabn {

constexpr float kLog2e = 1.44269504088896341f;

// 1/(1 + e^-x) and 1/(1 + e^x), its complement: both from t = e^-|x| <= 1, which cannot
// overflow.  Relative errors are a few ulps and, in the one that t multiplies, |x| * 2^-24
// from the rounding of the exponent's argument; a t below 2^-126 (|x| from 87.4 on) is taken
// as zero, so that SiLU is zero there (its value is below 1e-36).
__device__ __forceinline__ void sigmoids(float x, float& s, float& sc)
{
    const float t = __builtin_amdgcn_exp2f(-fabsf(x) * kLog2e);
    const float r = __builtin_amdgcn_rcpf(1.f + t);
    const float q = t * r;
    s = x >= 0.f ? r : q;
    sc = x >= 0.f ? q : r;
    if (x != x) s = sc = x;
}

// act(x) and act'(x).
template <int ACT>
__device__ __forceinline__ void glu_act(float x, float& f, float& d)
{
    if constexpr (ACT == kSilu) {
        float s, sc;
        sigmoids(x, s, sc);
        f = x * s;
        d = s * fmaf(x, sc, 1.f);
    } else if constexpr (ACT == kGelu) {
        const float P = 0.5f * erfcf(-x * 0.707106781186547524f);
        f = x * P;
        d = fmaf(x * 0.398942280401432678f, __builtin_amdgcn_exp2f(-0.5f * kLog2e * x * x), P);
    } else {
        const float k2 = 2.f * 0.797884560802865356f;         // 2 sqrt(2/pi)
        // s is 0 or 1 beyond |x| = 16, where x^3 may overflow
        const float y = x != x ? x : fminf(fmaxf(x, -16.f), 16.f);
        const float y2 = y * y;
        float s, sc;
        sigmoids(k2 * y * fmaf(0.044715f, y2, 1.f), s, sc);
        f = x * s;
        d = s * fmaf(y * sc, k2 * fmaf(0.134145f, y2, 1.f), 1.f);
    }
}

}  // namespace iabn
