// Activations of the feed-forward network and what their gradients need, in fp32.
#pragma once

#include <cuda_runtime.h>

namespace moonep {

// Values of moonep_activation (checked where the arguments are).
enum Act { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3, kActSwiglu = 4 };

// 1 / (1 + e^-x).  e^-x past fp32's range gives 0; the quotient's own flush (divisors of 2^126
// and more give 0) begins at x = -87.3, where the sigmoid is 1e-38.
__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + expf(-x)); }

// P(N(0,1) <= z), and e = exp(-z^2 / 2), sqrt(2 pi) times the density.
// For a = |z| the tail is e G(a), G(a) = erfcx(a / sqrt 2) / 2, and (1 + a / 2) G(a) is smooth in
// t = (a - 4) / (a + 4) over all of [0, inf) (the substitution of Shepherd and Laframboise, "Chebyshev
// approximation of (1 + 2x) exp(x^2) erfc x in 0 <= x < inf", 1981): a polynomial of degree 8, fitted
// to the smallest relative error (2.2e-8), one reciprocal for both quotients, and no branch.  What
// rounding a^2 takes from e is put back to first order: 5e-7 of the tail in fp32, where 1 + erf
// would cancel.  (erfcf, with a branch for each range, made the gelu epilogue of a tile of 128 x
// 256 take longer than its product at a depth of 1024.)  From a = 16 on e is 0.
__device__ __forceinline__ float normal_cdf(float z, float* density = nullptr) {
  const float a = fminf(fabsf(z), 16.f);
  const float s = a * a;
  float e = expf(-0.5f * s);
  e = fmaf(e, -0.5f * fmaf(a, a, -s), e);
  const float u = a + 4.f, v = fmaf(0.5f, a, 1.f);
  const float r = __fdividef(1.f, u * v);
  const float t = (a - 4.f) * v * r;
  float p = 2.554573875386e-04f;
  p = fmaf(p, t, 1.216406453750e-04f);
  p = fmaf(p, t, -2.259995089844e-03f);
  p = fmaf(p, t, 4.738154821098e-03f);
  p = fmaf(p, t, -6.626949179176e-04f);
  p = fmaf(p, t, -2.155544050038e-02f);
  p = fmaf(p, t, 6.918913871050e-02f);
  p = fmaf(p, t, -1.335505396128e-01f);
  p = fmaf(p, t, 2.832319140434e-01f);
  const float tail = e * p * (u * r);
  if (density != nullptr) *density = 0.3989422804f * e;
  return z > 0.f ? 1.f - tail : tail;
}

__device__ __forceinline__ float act_value(int act, float z) {
  if (act == kActRelu) return z < 0.f ? 0.f : z;  // (a NaN stays one)
  if (act == kActGelu) return z * normal_cdf(z);
  if (act == kActSilu) return z * sigmoid_f(z);
  return z;
}

// d act / d z at z
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if (ACT == kActRelu) return z > 0.f ? 1.f : (z <= 0.f ? 0.f : z);  // (a NaN stays one)
  if (ACT == kActGelu) {
    float density;
    const float c = normal_cdf(z, &density);
    return fmaf(z, density, c);
  }
  if (ACT == kActSilu) {
    const float s = sigmoid_f(z);
    return s * fmaf(z, 1.f - s, 1.f);
  }
  return 1.f;
}

}  // namespace moonep
