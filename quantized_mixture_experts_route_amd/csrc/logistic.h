// logistic.h -- the exponential and the logistic function in float32, to a few
// units, from the hardware's exponential and reciprocal.
#pragma once

#include "qmoe_device.h"

namespace qmoe {

// exp(-a) for a >= 0: the argument a log2(e) of the hardware's exponential is carried in two parts, since its
// rounding error would grow with a.  0 from 2^-150 on, and the hardware's 0 below 2^-126; NaN stays NaN.
__device__ inline float exp_minus(float a)
{
    constexpr float kLog2E = 1.44269502f, kLog2ERest = 1.92596299e-8f, kLn2 = 0.693147182f;
    const float hi = a * kLog2E, lo = fmaf(a, kLog2E, -hi) + a * kLog2ERest;
    return hi < 150.0f ? __builtin_amdgcn_exp2f(-hi) * fmaf(lo, -kLn2, 1.0f) : 0.0f * (a < INFINITY ? a : a == a ? 0.0f : a);
}

// exp(x) for x <= 0.
__device__ inline float exp_of(float x) { return exp_minus(-x); }

// s(z) = 1 / (1 + exp(-z)) and s(-z) = 1 - s(z).
struct Logistic {
    float s, rest;
};

__device__ inline Logistic logistic(float z)
{
    const float e = exp_minus(fabsf(z));
    const float d = 1.0f + e;
    float q = __builtin_amdgcn_rcpf(d);
    q = fmaf(fmaf(-d, q, 1.0f), q, q);
    const float eq = e * q;
    return z >= 0.0f ? Logistic{q, eq} : Logistic{eq, q};
}

}  // namespace qmoe
