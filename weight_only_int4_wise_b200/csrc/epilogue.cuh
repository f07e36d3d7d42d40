// The activation of the expert layer's up projection, applied in the GEMM
// epilogues (include/w4a16.h, W4A16_ACT_*).
#pragma once

#include <cuda_fp16.h>

#include "../../include/w4a16.h"

namespace w4a16 {

// Epilogue value: the fp32 accumulator rounded to fp16 (the product's result),
// then, for the expert layer's up projection, the activation evaluated in fp32
// on that fp16 value and rounded to fp16 again. GELU in both of its usual
// forms: x * Phi(x) with Phi the normal CDF (erf form), and the tanh
// approximation with the cubic term 0.044715 x^3. Both are written without
// the sum 1 + (something near -1) that loses all of fp32's digits for negative
// x: Phi(x) = erfc(-x / sqrt 2) / 2, and (1 + tanh u) / 2 = 1 / (1 + e^(-2u)).
__device__ __forceinline__ __half epilogue_value(float acc, int act) {
    const __half h = __float2half_rn(acc);
    if (act == W4A16_ACT_IDENTITY) return h;
    const float x = __half2float(h);
    float y;
    if (act == W4A16_ACT_RELU) {
        y = fmaxf(x, 0.f);
    } else if (act == W4A16_ACT_GELU_ERF) {
        y = 0.5f * x * erfcf(x * -0.70710678118654752f);
    } else {
        const float u = 0.79788456080286536f * (x + 0.044715f * x * x * x);
        y = x / (1.f + expf(-2.f * u));
    }
    return __float2half_rn(y);
}

// The gate's activation and its derivative, in fp32 on the unrounded
// projection (the gated product is rounded once, after the multiplication).
// As above, no value subtracts numbers near one: the normal CDF is erfc(-x / sqrt 2) / 2 and
// both the tanh GELU and SiLU are x * t with t = 1 / (1 + e^(-z)), z = 2 sqrt(2/pi) (x + 0.044715 x^3)
// or z = x, whose derivative is t + x t (1 - t) z'. (The derivative does subtract: from z = 17
// on 1 + e^(-z) and t are 1 and its second term 0, as the tests with the largest gates see;
// below, 1 - t is off by a few 2^-24, which x z' carries over: below 2^-16 of a derivative near
// one, against the 2^-11 of its rounding to fp16.)
// The logistic t uses the hardware exponential and division. By their published bounds (2 +
// floor(1.173 |z|) ulp and 2 ulp) the relative error of t is below 2^-17.6 where the result is
// not below fp16's range (|z| < 30), and below 2^-16.5 with the rounding of the tanh GELU's z,
// against the 2^-11 of its one rounding to fp16; they take 6 instead of about 25 instructions
// (the gated epilogue at 2048 x 14336 when it was changed: 482 -> 461 us).
constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhScale = 1.5957691216057308f;  // 2 sqrt(2 / pi)

__device__ __forceinline__ float logistic(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

__device__ __forceinline__ float gate_value(float x, int act) {
    switch (act) {
        case W4A16_ACT_SILU: return x * logistic(x);
        case W4A16_ACT_GELU_ERF: return 0.5f * x * erfcf(x * -kSqrtHalf);
        case W4A16_ACT_GELU_TANH: return x * logistic(kTanhScale * (x + 0.044715f * x * x * x));
        case W4A16_ACT_RELU: return x < 0.f ? 0.f : x;  // (fmaxf would turn a NaN into 0)
        default: return x;
    }
}

// The derivative, and the value in *v.
__device__ __forceinline__ float gate_slope(float x, int act, float* v) {
    switch (act) {
        case W4A16_ACT_SILU: {
            const float t = logistic(x);
            *v = x * t;
            return fmaf(x * t, 1.f - t, t);
        }
        case W4A16_ACT_GELU_ERF: {
            const float t = 0.5f * erfcf(x * -kSqrtHalf);
            *v = x * t;
            return fmaf(x * kInvSqrt2Pi, __expf(-0.5f * x * x), t);
        }
        case W4A16_ACT_GELU_TANH: {
            const float t = logistic(kTanhScale * (x + 0.044715f * x * x * x));
            *v = x * t;
            return fmaf(x * t * (1.f - t), kTanhScale * (1.f + 0.134145f * x * x), t);
        }
        case W4A16_ACT_RELU:
            *v = x < 0.f ? 0.f : x;
            return x > 0.f ? 1.f : (x <= 0.f ? 0.f : x);  // (a NaN's slope is that NaN, as for the other activations)
        default:
            *v = x;
            return 1.f;
    }
}

}  // namespace w4a16
