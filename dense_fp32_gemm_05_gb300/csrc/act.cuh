// Activations of the gated feed-forward operators, in fp32:
//
//   none  act(g) = g          silu  act(g) = g p,  p = 1 / (1 + exp(-v)), v = g
//   relu  act(g) = max(g, 0)  gelu  the same with v = 2 c (g + a g^3),
//                             c = sqrt(2 / pi), a = 0.044715: the tanh form, (1 + tanh(v / 2)) / 2 = p
//
// act'(g) = p (1 + g q v'(g)), q = 1 - p.  All from one exponential: with w = exp(v / 2) and
// r = 1 / (1 + w w), p = w (w r) and q = r, and act(g) = (g (w r)) w is right down to the
// smallest normal numbers, where p is none (with p = 1 / (1 + exp(-v)) it was 0 below
// v = -87.3).  NaN passes through (relu: 0 at NaN's derivative, as a comparison has it).
#pragma once

#include <cuda_runtime.h>

#include "../../include/sgemm_gb300.h"

namespace sgemm_gb300 {
namespace act {

inline bool is_activation(int a) { return a >= SGEMM_ACT_NONE && a <= SGEMM_ACT_GELU; }

// Of silu and gelu.  v and v' are taken of g cut to t: at silu's 60 and gelu's 8, where p is 1
// to the last bit, so that w w stays finite, and at gelu's -64, where p is 0, so that g^3 and
// t q v' do.  act(g) is within 2^-20 (1 + |v|) of it: the exponential's error grows with its
// argument, as does that of gelu's v.  ex2 and rcp are PTX's approximate ones: within 2^-22 each,
// and numbers that they flush to zero reach no result.  (With expf and a rounded quotient gated
// products of few rows took 0.2 to 0.4 us more.)
struct Parts {
    float w, wr, q, t, dv;

    template <int A>
    __device__ __forceinline__ static Parts of(float g) {
        constexpr float HALF = 0.72134752f;        // log2(e) / 2: w is 2 to HALF v
        constexpr float GELU = 1.5957691216057308f;    // 2 c
        Parts a;
        float half;
        if (A == SGEMM_ACT_GELU) {
            a.t = fmaxf(fminf(g, 8.0f), -64.0f);
            const float s = a.t * a.t;
            half = a.t * (GELU * HALF + GELU * HALF * 0.044715f * s);
            a.dv = GELU + GELU * 3.0f * 0.044715f * s;
        } else {
            a.t = fminf(g, 60.0f);
            half = HALF * a.t;
            a.dv = 1.0f;
        }
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a.w) : "f"(half));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a.q) : "f"(__fmaf_rn(a.w, a.w, 1.0f)));
        a.wr = a.w * a.q;
        return a;
    }
    __device__ __forceinline__ float value(float g) const { return g * wr * w; }
    // (1 is g 0 + 1: NaN where g is no finite number, as the formula is)
    __device__ __forceinline__ float slope(float g) const { return wr * w * __fmaf_rn(t * q, dv, __fmaf_rn(g, 0.0f, 1.0f)); }
};

template <int A>
__device__ __forceinline__ float value(float g) {
    if (A == SGEMM_ACT_NONE) return g;
    if (A == SGEMM_ACT_RELU) return g < 0.0f ? 0.0f : g;
    return Parts::of<A>(g).value(g);
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
    const Parts a = Parts::of<A>(g);
    slope = a.slope(g);
    return a.value(g);
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
