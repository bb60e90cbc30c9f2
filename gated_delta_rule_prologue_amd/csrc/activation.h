// activation.h -- the gate's activations and their slopes, shared by the gated norm and
// the short convolution.
#pragma once

#include "common.h"

namespace prism {

// e^-a for a >= 0 (a NaN stays one).  exp2 of the rounded product a log2 e is off by up to 64
// half steps of fp32 at a = 80.  That is nothing beside bf16's own rounding (2^-18 of the value
// against 2^-8); in fp32 it is 2^n 2^f with n + f = -a log2 e, |f| <= 1/2 and log2 e in two
// parts, so that f is rounded once and the error does not grow with a.
template <typename T> __device__ __forceinline__ float exp_minus(float a)
{
    if constexpr (sizeof(T) == 2)
        return __builtin_amdgcn_exp2f(a * -1.44269504088896341f);
    const float n = fmaxf(rintf(a * -1.44269504088896341f), -200.f);     // beyond it f takes the rest, and e^-a is zero
    const float f = __builtin_fmaf(a, -1.925962991e-8f, __builtin_fmaf(a, -1.44269502162933350f, -n));
    return ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
}

// act(z) and act'(z): s = 1 / (1 + e^-z) and c = 1 - s = 1 / (1 + e^z), both formed from
// e^-|z| <= 1 (a difference 1 - s would lose c of open gates: 6 % at z = 16, all of it from 18 on);
// silu = z s, silu' = s (1 + z c)
template <typename T, int GATE> __device__ __forceinline__ float gate_act(float z, float& slope)
{
    const float e = exp_minus<T>(fabsf(z)), d = __builtin_amdgcn_rcpf(1.f + e);
    const float s = z < 0.f ? e * d : d, c = z < 0.f ? d : e * d;
    if (GATE == 0) {
        slope = s * (1.f + z * c);
        return z * s;
    }
    slope = s * c;
    return s;
}

}  // namespace prism
