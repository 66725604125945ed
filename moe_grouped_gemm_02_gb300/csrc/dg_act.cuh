// The activations of the GEMM epilogues and of their backward pass, in FP32.
#pragma once

#include "dg_internal.h"

namespace dg {

__device__ __forceinline__ float ex2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / (1 + e^-x).  The approximate 2^x and reciprocal are good to a few FP32 rounding steps (the
// product with log2 e adds ~1e-6 at |x| = 20, where the result or its distance from 1 is below 2e-9), far below the
// BF16 rounding of D, z and dz; a large -x gives 0, a large x 1.  The FP32 bias gradient sums slopes computed
// from it: over all BF16 z up to 60 they are off by at most 2^-23.1 (silu), 2^-21.3 (gelu), 2^-23.0 (swiglu) of
// max(1, |z|), as much as with expf and a division in FP32 (2^-23.1, 2^-21.3, 2^-23.0).
constexpr float LOG2E = 1.4426950408889634f;
__device__ __forceinline__ float act_sigmoid(float x) { return rcp_approx(1.0f + ex2_approx(-LOG2E * x)); }

constexpr float GELU_C = 0.7978845608028654f;    // sqrt(2 / pi)
constexpr float GELU_D = 0.044715f;

// h = act(v) for the activations that act on one value.  gelu is the tanh form:
// 0.5 (1 + tanh u) = sigmoid(2u), u = sqrt(2/pi) (v + 0.044715 v^3).
template <int ACT>
__device__ __forceinline__ float act_one(float v) {
    if constexpr (ACT == ACT_RELU) return v > 0.0f ? v : (v != v ? v : 0.0f);
    if constexpr (ACT == ACT_GELU) return v * act_sigmoid(2.0f * GELU_C * (v + GELU_D * v * v * v));
    if constexpr (ACT == ACT_SILU) return v * act_sigmoid(v);
    return v;
}

// The larger of two values; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Two values of an activation.  silu and gelu, v sigmoid(a), share one reciprocal between the two: with
// e = 2^(-a log2 e), 1/(1 + e0) = (1 + e1) / ((1 + e0)(1 + e1)), so a value costs one and a half
// operations of the special function unit, which bounds the epilogue of a tile with a short K, instead of
// two.  e is held at 2^62, so that the product stays finite, and v at -43 in the result: below a = -43, where
// |act| < 1e-17, the result is -1e-17 at most instead of smaller still.  (A value's last FP32 bits depend on the other
// one's through the shared rounding: D may be the next BF16 value.)
template <int ACT>
__device__ __forceinline__ void act_two(float v0, float v1, float& h0, float& h1) {
    if constexpr (ACT == ACT_SILU || ACT == ACT_GELU) {
        constexpr float S = ACT == ACT_SILU ? -LOG2E : -2.0f * GELU_C * LOG2E;
        const float a0 = ACT == ACT_SILU ? v0 : v0 + GELU_D * v0 * v0 * v0;
        const float a1 = ACT == ACT_SILU ? v1 : v1 + GELU_D * v1 * v1 * v1;
        const float d0 = 1.0f + ex2_approx(fminf(S * a0, 62.0f)), d1 = 1.0f + ex2_approx(fminf(S * a1, 62.0f));
        const float r = rcp_approx(d0 * d1);
        h0 = max_nan(v0, -43.0f) * (r * d1);
        h1 = max_nan(v1, -43.0f) * (r * d0);
    } else {
        h0 = act_one<ACT>(v0);
        h1 = act_one<ACT>(v1);
    }
}

// The gated pair: silu(gate) * up.
__device__ __forceinline__ float act_swiglu(float gate, float up) { return gate * act_sigmoid(gate) * up; }

// d act(v) / dv.
template <int ACT>
__device__ __forceinline__ float act_slope(float v) {
    if constexpr (ACT == ACT_RELU) return v > 0.0f ? 1.0f : (v != v ? v : 0.0f);
    if constexpr (ACT == ACT_GELU) {
        const float t = act_sigmoid(2.0f * GELU_C * (v + GELU_D * v * v * v));
        // (v * v is held below overflow: t (1 - t) is 0 long before)
        return t + v * (t - t * t) * (2.0f * GELU_C + 6.0f * GELU_C * GELU_D * fminf(v * v, 1e30f));
    }
    if constexpr (ACT == ACT_SILU) {
        const float t = act_sigmoid(v);
        return t * (1.0f + v * (1.0f - t));
    }
    return 1.0f;
}

}  // namespace dg
