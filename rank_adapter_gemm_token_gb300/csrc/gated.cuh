// The activations of a gated feed-forward block, in fp32.
#pragma once
#include "mlora.h"

namespace mlora {

// g / (1 + e^-x): the silu with x = g, and the tanh form of the gelu with x = 2 sqrt(2 / pi) (g + 0.044715 g^3), since
// (1 + tanh(x / 2)) / 2 = 1 / (1 + e^-x). Far to the left e^-x is infinite and the quotient the -0 that it tends to.
__device__ __forceinline__ float gate_sigmoid(float g, float x) { return __fdividef(g, 1.0f + __expf(-x)); }

// erfc and not 1 + erf: to the left of 0 the sum would cancel.
__device__ __forceinline__ float gate(float g, int act) {
  if (act == MLORA_ACT_SILU) return gate_sigmoid(g, g);
  if (act == MLORA_ACT_GELU_TANH) return gate_sigmoid(g, g * fmaf(0.07135481627f, g * g, 1.5957691216f));
  return 0.5f * g * erfcf(-0.70710678119f * g);
}

}  // namespace mlora
