// The gated scan's gates, shared by its forward, gradient and step.
//
// With s = sigmoid(forget) a token moves a channel's state by h = a h + w v x,
// where v = sigmoid(input_gate) (1 without one) and
//   without rates  a = s, w = 1 - s                        (a convex average),
//   with a rate r  p = r s, a = exp(-p), w = sqrt(1 - a^2)  (a normalised one).
// A rate below 0 counts as 0: the state is held and takes no input.
#pragma once

#include "sequence.hpp"

namespace sca {

// sigmoid(v) and sigmoid(-v).  The greater one is within a few units of its last place,
// the smaller within (|v| + 8) 2^-24 of itself, as the exponent's product is rounded; 1
// minus a rounded sigmoid would lose its digits altogether.
struct Sides { float up, down; };
__device__ __forceinline__ Sides sides(float v) {
  const float e = exp2_hw(-__builtin_fabsf(v) * kLog2e);   // in (0, 1]
  const float r = rcp_hw(1.0f + e), er = e * r;
  return v >= 0.0f ? Sides{r, er} : Sides{er, r};
}

// 1 - 4^l for l <= 0, 4^l = q being known.  Above -0.36 (q above 0.6), where the
// difference loses digits, a polynomial (least maximum of the relative error of its quotient
// by l, 9e-8, fitted there) that in float32 is within 2e-7 of it.
__device__ __forceinline__ float one_minus_4(float l, float q) {
  float s = __builtin_fmaf(l, -0.0346682966f, -0.151432544f);
  s = __builtin_fmaf(l, s, -0.443717122f);
  s = __builtin_fmaf(l, s, -0.960891604f);
  s = __builtin_fmaf(l, s, -1.38629425f);
  s *= l;
  materialize(s);                            // a select, not a branch around the polynomial
  return l > -0.36067376f ? s : 1.0f - q;
}

// What a token's gate does: decay a, log2 of it, the input's weight w.
struct Gate { float a, log_a, w; };

// nr: -log2(e) times the rate, at most 0 (unused without rates).
template <bool RATE>
__device__ __forceinline__ Gate gate(float forget, float nr) {
  Gate g;
  if constexpr (RATE) {
    g.log_a = nr * sigmoid(forget);
    g.a = exp2_hw(g.log_a);
    g.w = __builtin_amdgcn_sqrtf(one_minus_4(g.log_a, g.a * g.a));
  } else {
    const Sides s = sides(forget);
    g.a = s.up;
    g.w = s.down;
    // log2 sigmoid(v) = min(v, 0) log2(e) - log2(1 + exp(-|v|))
    g.log_a = __builtin_amdgcn_logf(s.up);
  }
  return g;
}

// -log2(e) r of a rate, a negative one counting as 0 and an infinite one as 1e38, so
// that a closed gate (s = 0) holds the state under any rate (a NaN stays one).
__device__ __forceinline__ float rate_log2(float r) {
  return at_most(at_least(r, 0.0f), 1e38f) * -kLog2e;
}

}  // namespace sca
