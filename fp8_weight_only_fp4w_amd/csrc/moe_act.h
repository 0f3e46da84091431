// Activations of an expert's gate, shared by the mixture-of-experts kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "device.h"

namespace fp4w {

// act(gate) * up in FP32 (kind: fp4w_activation).
//   silu(g) = g / (1 + exp(-g));  gelu(g) = g / (1 + exp(-2 z)), z = sqrt(2 / pi) (g + 0.044715 g^3),
// the tanh form of gelu: 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z)).  A gate far below zero gives
// exp = inf and so the limit 0.
__device__ __forceinline__ float gated(int kind, float g, float up) {
  const float z = kind == 0 ? g : 1.5957691216057308f * fmaf(0.044715f * g * g, g, g);
  return g / (1.0f + expf(-z)) * up;
}

}  // namespace fp4w
