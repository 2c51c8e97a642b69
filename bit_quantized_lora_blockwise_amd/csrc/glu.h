// The gated activation H = silu(G) U and its gradients, in fp32.
#pragma once

#include "common.h"

namespace glu {

// 1 / (1 + e^-g): exp2 and the reciprocal are off by about one unit in the last place each,
// which the rounding of H to bf16 does not see and that of gradients in fp32 takes as it
// takes the sums'.  For g below -88 the exponential is infinite and the result 0, as in the limit.
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.442695041f * g));
}

__device__ __forceinline__ float silu(float g) { return g * sigmoid(g); }

// dG = dH U sig (1 + G (1 - sig)), dU = dH G sig
__device__ __forceinline__ void back(float g, float u, float dh, float& dg, float& du) {
  const float s = sigmoid(g), gs = g * s;
  du = dh * gs;
  dg = dh * u * fmaf(gs, 1.0f - s, s);
}

}  // namespace glu
