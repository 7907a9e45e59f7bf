// block_math.cuh -- the gated block's activations and their derivatives on
// fp32 values.
#pragma once

#include "block_params.h"
#include "epilogue_math.cuh"

namespace spgemm {

// Logistic function.  __expf overflows to +inf for g < -88 and the quotient
// is then 0, its limit.
__device__ __forceinline__ float logistic(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// act(g): SiLU g / (1 + e^-g), tanh-GELU (the epilogue's form) or ReLU.
// __fdividef(x, y) is 0 for y above 2^126, so SiLU and GELU of a very
// negative g are -0, their limit.
template <int ACT>
__device__ __forceinline__ float gate_act(float g) {
  if constexpr (ACT == kActSilu) return __fdividef(g, 1.0f + __expf(-g));
  if constexpr (ACT == kActGelu) return gelu_tanh(g);
  return g > 0.0f ? g : (g != g ? g : 0.0f);  // ReLU; NaN stays NaN
}

// a = act(g) and d = act'(g).
//   SiLU: s = logistic(g); a = g s; a' = s (1 + g (1 - s)) = s + a (1 - s)
//   GELU: with s = logistic(2u), u = c (g + k g^3): a = g s (since
//         (1 + tanh u) / 2 = s), a' = s + a (1 - s) 2u', 2u' = 2c (1 + 3k g^2)
//   ReLU: a' = [g > 0]
// g = +-inf is left to IEEE arithmetic, as the formula evaluated term by term.
template <int ACT>
__device__ __forceinline__ void gate_act_grad(float g, float& a, float& d) {
  if constexpr (ACT == kActRelu) {
    a = gate_act<kActRelu>(g);
    d = g > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kActSilu) {
    const float s = logistic(g);
    a = g * s;
    d = fmaf(a, 1.0f - s, s);
  } else {
    const float g2 = g * g;
    const float s = logistic(1.5957691216f * g * fmaf(0.044715f, g2, 1.0f));
    a = g * s;
    // Where a (1 - s) is 0 the second term is 0 in the limit, but g^2 may
    // have overflowed: no 0 x inf.
    const float t = a * (1.0f - s);
    d = t == 0.0f ? s : fmaf(t, 1.5957691216f * fmaf(3.0f * 0.044715f, g2, 1.0f), s);
  }
}

}  // namespace spgemm
