// The activations of the gated feed-forward block: act(a) = a s(z(a)) with the logistic function s.
#pragma once
#include "common.hpp"
#include "ffn.hpp"

namespace moe {
namespace ffn {

// SiLU z = a; GELU (tanh form) z = 2 sqrt(2 / pi) (a + 0.044715 a^3)
constexpr float kZ1 = 1.5957691216057308f, kZ3 = 1.5957691216057308f * 0.044715f;
template <int ACT>
__device__ __forceinline__ float act(float a) {
  return a * sigmoidf_(ACT == kSilu ? a : a * (kZ1 + kZ3 * a * a));
}
// act(a) and act'(a) = s + a s (1 - s) z'(a).  Where a^2 is past 256, s is 0 or 1 and the second term 0, whose last
// factor must not overflow.
template <int ACT>
__device__ __forceinline__ void act_grad(float a, float& f, float& d) {
  const float s = sigmoidf_(ACT == kSilu ? a : a * (kZ1 + kZ3 * a * a));
  f = a * s;
  d = s + f * (1.0f - s) * (ACT == kSilu ? 1.0f : kZ1 + 3.0f * kZ3 * fminf(a * a, 256.0f));
}

}  // namespace ffn
}  // namespace moe
