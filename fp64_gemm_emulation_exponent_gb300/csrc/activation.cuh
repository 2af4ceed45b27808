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

// From e^-|z|, which never leaves fp32's range on the large side: 1 / (1 + e^-z)
// is 0 from z = -87.3 on, where __fdividef's divisor passes 2^126, though the
// function is 2^-126 there and act(g) u need not be small.
__device__ __forceinline__ float act_logistic(float z) {
  const float t = __expf(-fabsf(z)), r = __fdividef(1.0f, 1.0f + t);
  return z < 0.0f ? t * r : r;
}

constexpr float kGeluA = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f * kGeluA;

// The normal distribution's tail beyond |g|, e^(-g^2/2) t p(t) with t = 1 / (1 +
// 0.3 |g|): what the exponential leaves is smooth in t, and p, of degree 7, is
// fitted to it for 0 <= |g| <= 14 by least squares at Chebyshev's points,
// reweighted towards the largest relative error (1.7e-7; 5e-7 in fp32, the
// exponential aside).  With erfcf in its place the epilogue of a product with
// gelu cost 3.5 us more on 1999 rows, 1032 -> 520, and 30 of 180 on 8192 rows,
// 4096 -> 2048: its instructions slow the warps that issue copies and MMAs.
__device__ __forceinline__ float normal_tail(float g) {
  const float t = __fdividef(1.0f, fmaf(0.3f, fabsf(g), 1.0f));
  float p = 0.03567477688193321f;
  p = fmaf(p, t, -0.15720310807228088f);
  p = fmaf(p, t, 0.20635353028774261f);
  p = fmaf(p, t, -0.05368367210030556f);
  p = fmaf(p, t, 0.12856164574623108f);
  p = fmaf(p, t, 0.09991348534822464f);
  p = fmaf(p, t, 0.12075395882129669f);
  p = fmaf(p, t, 0.11962930113077164f);
  return __expf(-0.5f * g * g) * (t * p);
}

__device__ __forceinline__ float act_p(float g, int act) {
  if (act == OZK_SILU) return act_logistic(g);
  if (act == OZK_GELU_TANH) return act_logistic(g * fmaf(kGeluB, g * g, kGeluA));
  const float tail = normal_tail(g);
  return g < 0.0f ? tail : 1.0f - tail;
}
// act(g) within a few units of 2^-23, for results in fp32: silu 4, gelu 5.5,
// gelu_tanh 4 + 2 |z|, where the forms above are off by up to 12 + 2.7 |z| with z
// the exponential's argument.  An epilogue of a few rows takes few values, and the
// functions in full cost it 0.1 us (1 x 2 x 8192 x 4096 NVFP4 10.7 -> 10.8).
__device__ __forceinline__ float act_value(float g, int act) {
  if (act == OZK_GELU) return g * normcdff(g);
  const float z = act == OZK_SILU ? g : g * fmaf(kGeluB, g * g, kGeluA);
  const float t = expf(-fabsf(z)), r = __frcp_rn(1.0f + t);
  return g * (z < 0.0f ? t * r : r);
}

// The derivative g P'(g) + P(g), given P(g).
__device__ __forceinline__ float act_slope(float g, float p, int act) {
  if (act == OZK_SILU) return fmaf(g * p, 1.0f - p, p);
  // g^2 held finite: beside it 1 - p or p is 0
  if (act == OZK_GELU_TANH) return fmaf(g * p * (1.0f - p), fmaf(3.0f * kGeluB, fminf(g * g, 1e30f), kGeluA), p);
  return fmaf(g * 0.39894228040143268f, __expf(-0.5f * g * g), p);
}

}  // namespace
}  // namespace ozk
