// zero_act.h -- the activations of the linear operators and their slopes, in fp32.
#pragma once

#include <hip/hip_runtime.h>

#include "zero.h"

#pragma clang fp contract(off)

namespace zk {
namespace act {

// exp(x^2) erfc(x), x >= 0: a polynomial in t = 1 / (1 + 0.37 x) without constant
// term, fitted to the relative error by reweighted least squares; within 1.2e-6
// where exp(-x^2) is a normal number.
__device__ __forceinline__ float erfcx(float x) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.37f, x, 1.0f));
  float s = -0.1425526887178421f;
  s = __builtin_fmaf(s, t, 0.43566352128982544f);
  s = __builtin_fmaf(s, t, -0.18643616139888763f);
  s = __builtin_fmaf(s, t, 0.31740835309028625f);
  s = __builtin_fmaf(s, t, 0.15265494585037231f);
  s = __builtin_fmaf(s, t, 0.21488286554813385f);
  s = __builtin_fmaf(s, t, 0.208379864692688f);
  return s * t;
}

constexpr float kLog2e = 1.44269504f;
constexpr float kRoot2OverPi = 0.797884561f, kCubic = 0.044715f;

__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// The standard normal's distribution function, and exp(-z^2 / 2).  The lower tail
// keeps its relative accuracy.
__device__ __forceinline__ float phi(float z, float& e) {
  const float a = __builtin_fabsf(z);
  e = __builtin_amdgcn_exp2f(-0.72134752f * (z * z));
  const float tail = 0.5f * erfcx(0.70710678f * a) * e;
  return z > 0.0f ? 1.0f - tail : tail;
}

// At the far negative end gelu and silu are their limit, 0; NaN stays NaN.
__device__ __forceinline__ float forward(int kind, float z) {
  if (kind == ZERO_ACT_NONE) return z;
  if (kind == ZERO_ACT_RELU) return z < 0.0f ? 0.0f : z;
  const float w = z < -128.0f ? -128.0f : z;
  if (kind == ZERO_ACT_GELU) {
    float e;
    const float p = phi(w, e);
    return w * p;
  }
  if (kind == ZERO_ACT_GELU_TANH) return w * sigmoid(2.0f * kRoot2OverPi * w * __builtin_fmaf(kCubic * w, w, 1.0f));
  return w * sigmoid(w);
}

// d act / dz.  Beyond +-128 the slopes are 0 and 1 in fp32.
__device__ __forceinline__ float slope(int kind, float z) {
  if (kind == ZERO_ACT_NONE) return 1.0f;
  if (kind == ZERO_ACT_RELU) return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;
  const float w = __builtin_fabsf(z) > 128.0f ? __builtin_copysignf(128.0f, z) : z;
  if (kind == ZERO_ACT_GELU) {
    float e;
    const float p = phi(w, e);
    return __builtin_fmaf(0.398942280f * w, e, p);
  }
  if (kind == ZERO_ACT_GELU_TANH) {
    const float w2 = w * w;
    const float s = sigmoid(2.0f * kRoot2OverPi * w * __builtin_fmaf(kCubic, w2, 1.0f));
    return __builtin_fmaf(w * s * (1.0f - s), 2.0f * kRoot2OverPi * __builtin_fmaf(3.0f * kCubic, w2, 1.0f), s);
  }
  const float s = sigmoid(w);
  return s * __builtin_fmaf(w, 1.0f - s, 1.0f);
}

}  // namespace act
}  // namespace zk
