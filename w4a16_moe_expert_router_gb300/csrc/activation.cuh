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

// The activation y and its derivative dy at z, for the gradient, where both are wanted for
// every element and their arithmetic, not memory, would be the bound: one exponential each.
// With p = s(v): d(z p)/dz = p + z p (1 - p) v', and e = e^-|v| gives p and 1 - p = s(-v)
// without cancellation.  The erf form takes erfc(x) = t (a1 + t (a2 + .. a5)) e^(-x^2), t = 1 /
// (1 + 0.3275911 x), x >= 0 (Abramowitz and Stegun 7.1.26, off by 1.5e-7 at most), whose
// exponential is the normal density's too: d(z c)/dz = c + z e^(-z^2 / 2) / sqrt(2 pi).
__device__ __forceinline__ void activate_grad(float z, int act, float& y, float& dy) {
  if (act == kIdentity) {
    y = z;
    dy = 1.f;
    return;
  }
  if (act == kGeluErf) {
    const float x = 0.70710678118654752f * fabsf(z), e = __expf(-x * x);
    const float t = __fdividef(1.f, fmaf(0.3275911f, x, 1.f));
    const float half =
        0.5f * e * t *
        fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f), 0.254829592f);
    const float c = z < 0.f ? half : 1.f - half;  // erfc(-z / sqrt 2) / 2
    y = z * c;
    dy = e == 0.f ? c : fmaf(0.39894228040143268f * z, e, c);  // far out z may be infinite
    return;
  }
  const float z2 = z * z;
  const float v = act == kSilu ? z : kTwoRootTwoOverPi * z * fmaf(0.044715f, z2, 1.f);
  const float dv = act == kSilu ? 1.f : kTwoRootTwoOverPi * fmaf(3.f * 0.044715f, z2, 1.f);
  const float e = __expf(-fabsf(v)), r = __fdividef(1.f, 1.f + e), er = e * r;
  const float p = v < 0.f ? er : r, pq = r * er;
  y = z * p;
  // p (1 - p) falls faster than v' grows, but far out the product would be 0 times inf
  dy = pq == 0.f ? p : fmaf(z * pq, dv, p);
}

}  // namespace moe
