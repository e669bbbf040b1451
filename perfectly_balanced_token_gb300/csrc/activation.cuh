// Activations of the feed-forward network and their gradients, in fp32.
#pragma once

#include <cuda_runtime.h>

namespace moonep {

// Values of moonep_activation (checked where the arguments are).
enum Act { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3, kActSwiglu = 4 };

// 1 / (1 + e^-x).  e^-x past fp32's range gives 0; the quotient's own flush (divisors of 2^126
// and more give 0) begins at x = -87.3, where the sigmoid is 1e-38.
__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + expf(-x)); }

// P(N(0,1) <= x) through erfc, which keeps its relative accuracy where 1 + erf cancels.
__device__ __forceinline__ float normal_cdf(float x) { return 0.5f * erfcf(x * -0.70710678f); }

__device__ __forceinline__ float act_value(int act, float z) {
  if (act == kActRelu) return z < 0.f ? 0.f : z;  // (a NaN stays one)
  if (act == kActGelu) return z * normal_cdf(z);
  if (act == kActSilu) return z * sigmoid_f(z);
  return z;
}

}  // namespace moonep
