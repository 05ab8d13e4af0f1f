// Activations of the gated feed-forward operators, in fp32:
//
//   none  act(g) = g          silu  act(g) = g p,  p = 1 / (1 + exp(-g))
//   relu  act(g) = max(g, 0)  gelu  act(g) = g p,  p = 1 / (1 + exp(-v)), v = 2 c (g + a g^3),
//                             c = sqrt(2 / pi), a = 0.044715: the tanh form, (1 + tanh(v / 2)) / 2 = p
//
// act(g) = factor * g, and act'(g) = p (1 + g (1 - p) v'(g)): both from one exponential (and in
// gelu's from g cut to +-64, where p is 0 or 1: with a finite g past 4e35 its second term was
// 0 times an infinity).
// NaN passes through (relu: 0 at NaN's derivative, as a comparison has it).
#pragma once

#include <cuda_runtime.h>

#include "../../include/sgemm_gb300.h"

namespace sgemm_gb300 {
namespace act {

inline bool is_activation(int a) { return a >= SGEMM_ACT_NONE && a <= SGEMM_ACT_GELU; }

// p, v'(g) and the g that both are of (t), of silu and gelu.  gelu takes v from g cut to +-64, where p is 0 or 1 to
// the last bit: g^3 and v' stay finite.  __expf's error is 2 units and a few more as its
// argument grows; where that counts p is far below a bf16 unit of 1.
template <int A>
__device__ __forceinline__ float factor_of(float g, float &t, float &dv) {
    float v = g;
    t = g;
    dv = 1.0f;
    if (A == SGEMM_ACT_GELU) {
        t = fabsf(g) > 64.0f ? copysignf(64.0f, g) : g;
        const float s = t * t;
        v = 1.5957691216057308f * t * (1.0f + 0.044715f * s);
        dv = 1.5957691216057308f * (1.0f + 0.134145f * s);
    }
    return __fdividef(1.0f, 1.0f + __expf(-v));
}

template <int A>
__device__ __forceinline__ float value(float g) {
    if (A == SGEMM_ACT_NONE) return g;
    if (A == SGEMM_ACT_RELU) return g < 0.0f ? 0.0f : g;
    float t, dv;
    return g * factor_of<A>(g, t, dv);
}

// act(g), and its derivative.
template <int A>
__device__ __forceinline__ float value_slope(float g, float &slope) {
    if (A == SGEMM_ACT_NONE) {
        slope = 1.0f;
        return g;
    }
    if (A == SGEMM_ACT_RELU) {
        slope = g > 0.0f ? 1.0f : 0.0f;
        return g < 0.0f ? 0.0f : g;
    }
    float t, dv;
    const float p = factor_of<A>(g, t, dv);
    slope = p * (1.0f + t * (1.0f - p) * dv);
    return g * p;
}

// f(A) with the activation as a constant.  A loop over many values belongs inside f: with a
// branch at each value their exponentials and quotients, ~150 clocks one after
// the other, do not overlap.
template <int A>
struct Constant {
    static constexpr int value = A;
};
template <typename Fn>
__device__ __forceinline__ void with(int a, Fn f) {
    if (a == SGEMM_ACT_SILU) f(Constant<SGEMM_ACT_SILU>());
    else if (a == SGEMM_ACT_GELU) f(Constant<SGEMM_ACT_GELU>());
    else if (a == SGEMM_ACT_RELU) f(Constant<SGEMM_ACT_RELU>());
    else f(Constant<SGEMM_ACT_NONE>());
}

}  // namespace act
}  // namespace sgemm_gb300
