// Activations of the gated products and their derivatives, in fp32.
//
// Each is g P(g) with P rising from 0 to 1: the logistic function (silu), the
// normal distribution's (gelu), or the latter's approximation (1 + tanh z) / 2
// with z = sqrt(2 / pi) (g + 0.044715 g^3), the logistic function of 2 z
// (gelu_tanh).  In this form nothing cancels for large negative g.
#pragma once

#include <cuda_runtime.h>

#include "ozk.h"

namespace ozk {
namespace {

__device__ __forceinline__ float act_logistic(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

constexpr float kGeluA = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f * kGeluA;

__device__ __forceinline__ float act_p(float g, int act) {
  if (act == OZK_SILU) return act_logistic(g);
  if (act == OZK_GELU_TANH) return act_logistic(g * fmaf(kGeluB, g * g, kGeluA));
  return 0.5f * erfcf(g * -0.70710678118654752f);
}
__device__ __forceinline__ float act_value(float g, int act) { return g * act_p(g, act); }

// The derivative g P'(g) + P(g), given P(g).
__device__ __forceinline__ float act_slope(float g, float p, int act) {
  if (act == OZK_SILU) return fmaf(g * p, 1.0f - p, p);
  // g^2 held finite: beside it 1 - p or p is 0
  if (act == OZK_GELU_TANH) return fmaf(g * p * (1.0f - p), fmaf(3.0f * kGeluB, fminf(g * g, 1e30f), kGeluA), p);
  return fmaf(g * 0.39894228040143268f, __expf(-0.5f * g * g), p);
}

}  // namespace
}  // namespace ozk
