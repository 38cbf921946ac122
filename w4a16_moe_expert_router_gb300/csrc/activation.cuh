// activation.cuh -- the activations of the 16-bit layer's products and their derivatives.
#pragma once

#include <cstdint>

namespace moe {

constexpr int kGeluTanh = 0, kGeluErf = 1, kSilu = 2, kIdentity = 3;

// 1 / (1 + e^-v), finite for every v (e^-v = inf gives 0)
__device__ __forceinline__ float logistic(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// GELU's tanh form is z s(2 y), s the logistic function, y = sqrt(2 / pi) (z + 0.044715 z^3),
// since (1 + tanh y) / 2 = s(2 y).  The erf form uses the complementary error function,
// z erfc(-z / sqrt 2) / 2, which keeps its digits where 1 + erf would cancel.
constexpr float kTwoRootTwoOverPi = 1.59576912160573071f;
__device__ __forceinline__ float activate(float z, int act) {
  if (act == kGeluTanh) return z * logistic(kTwoRootTwoOverPi * z * fmaf(0.044715f * z, z, 1.f));
  if (act == kGeluErf) return 0.5f * z * erfcf(-0.70710678118654752f * z);
  if (act == kSilu) return z * logistic(z);
  return z;
}

// The activation y and its derivative dy at z.  With p = s(v): d(z p)/dz = p + z p (1 - p) v',
// 1 - p = s(-v) without cancellation; the erf form's derivative adds z times the normal density.
__device__ __forceinline__ void activate_grad(float z, int act, float& y, float& dy) {
  if (act == kIdentity) {
    y = z;
    dy = 1.f;
    return;
  }
  if (act == kGeluErf) {
    const float c = 0.5f * erfcf(-0.70710678118654752f * z);
    y = z * c;
    dy = fmaf(0.39894228040143268f * z, __expf(-0.5f * z * z), c);
    return;
  }
  const float z2 = z * z;
  const float v = act == kSilu ? z : kTwoRootTwoOverPi * z * fmaf(0.044715f, z2, 1.f);
  const float dv = act == kSilu ? 1.f : kTwoRootTwoOverPi * fmaf(3.f * 0.044715f, z2, 1.f);
  const float p = logistic(v), q = logistic(-v);
  y = z * p;
  // p q falls faster than dv grows, but either may be 0 times inf far out, where the term is 0
  const float w = z * (p * q) * dv;
  dy = p + (p * q == 0.f ? 0.f : w);
}

}  // namespace moe
