// Activations of the feed-forward network and what their gradients need, in fp32, two values at a
// time: the epilogues and the gradient kernels are bound by instructions where they are not by
// memory, and one packed instruction (fma.rn.f32x2 and its kin) serves both values.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moonep {

// Values of moonep_activation (checked where the arguments are).
enum Act { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3, kActSwiglu = 4 };

// ---- two fp32 values ----------------------------------------------------------
struct F2 {
  uint64_t bits;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ explicit F2(float x) : F2(x, x) {}
  __device__ __forceinline__ F2(float x, float y) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(bits) : "f"(x), "f"(y));
  }
  __device__ __forceinline__ void get(float& x, float& y) const {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(bits));
  }
};
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.bits) : "l"(a.bits), "l"(b.bits));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.bits) : "l"(a.bits), "l"(b.bits));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.bits) : "l"(a.bits), "l"(b.bits), "l"(c.bits));
  return r;
}
// 2^x and 1/x by the special-function unit (PTX: relative errors of 2^-22 and 2^-23)
__device__ __forceinline__ F2 exp2_2(F2 a) {
  float x, y;
  a.get(x, y);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(y));
  return F2(x, y);
}
__device__ __forceinline__ F2 recip2(F2 a) {
  float x, y;
  a.get(x, y);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(y));
  return F2(x, y);
}

// 1 / (1 + e^-z).  The product z log2 e is rounded, so e^-z is off by up to 2^-24 |z| of itself: 1e-6
// of a sigmoid of e^-17.  e^-z past fp32's range gives 0, and so do sums of 2^126 and more (z below
// -87.3, where the sigmoid is 1e-38).
__device__ __forceinline__ F2 sigmoid2(F2 z) {
  return recip2(F2(1.f) + exp2_2(z * F2(-1.4426950408889634f)));
}

// P(N(0,1) <= z), and the density.
// For a = |z| the tail is e G(a), e = exp(-a^2 / 2), G(a) = erfcx(a / sqrt 2) / 2, and (a + k) G(a) is
// smooth in t = (a - k) / (a + k) = 1 - 2k / (a + k) over all of [0, inf) (the substitution of Shepherd
// and Laframboise, "Chebyshev approximation of (1 + 2x) exp(x^2) erfc x in 0 <= x < inf", 1981):
// with k = 4.25 a polynomial of degree 7, fitted to the smallest relative error (1.2e-7), one
// reciprocal and no branch, where 1 + erf would cancel.  Roundings of a^2 and of the exponent make
// it 2^-24 a^2 of the tail more.  (erfcf, with a branch for each range, made the gelu epilogue of a
// tile take several times as long as its product.)  From a = 16 on e is 0.
__device__ __forceinline__ F2 normal_cdf2(F2 z, F2* density = nullptr) {
  float x, y;
  z.get(x, y);
  const F2 a(fminf(fabsf(x), 16.f), fminf(fabsf(y), 16.f));
  const F2 e = exp2_2(a * a * F2(-0.72134752044448170f));
  const F2 r = recip2(a + F2(4.25f));
  const F2 t = fma2(r, F2(-8.5f), F2(1.f));
  F2 p(2.106905449182e-03f);
  p = fma2(p, t, F2(-1.038260525092e-03f));
  p = fma2(p, t, F2(-1.938312128186e-02f));
  p = fma2(p, t, F2(8.534678816795e-02f));
  p = fma2(p, t, F2(-2.205096930265e-01f));
  p = fma2(p, t, F2(4.182209968567e-01f));
  p = fma2(p, t, F2(-6.251299977303e-01f));
  p = fma2(p, t, F2(7.595543265343e-01f));
  const F2 tail = e * r * p;
  if (density != nullptr) *density = e * F2(0.3989422804f);
  float tx, ty, cx, cy;
  tail.get(tx, ty);
  fma2(tail, F2(-1.f), F2(1.f)).get(cx, cy);
  return F2(x > 0.f ? cx : tx, y > 0.f ? cy : ty);
}

// ---- the activations ----------------------------------------------------------
template <int ACT>
__device__ __forceinline__ F2 act2(F2 z) {
  if (ACT == kActRelu) {
    float x, y;
    z.get(x, y);
    return F2(x < 0.f ? 0.f : x, y < 0.f ? 0.f : y);  // (a NaN stays one)
  }
  if (ACT == kActGelu) return z * normal_cdf2(z);
  if (ACT == kActSilu) return z * sigmoid2(z);
  return z;
}

// act of N values, N even
template <int ACT, int N>
__device__ __forceinline__ void act_each(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) act2<ACT>(F2(v[i], v[i + 1])).get(v[i], v[i + 1]);
}
template <int N>
__device__ __forceinline__ void act_each(int act, float (&v)[N]) {  // one loop for each activation
  if (act == kActRelu) act_each<kActRelu>(v);
  else if (act == kActGelu) act_each<kActGelu>(v);
  else if (act == kActSilu) act_each<kActSilu>(v);
}
// v = silu(v) u
template <int N>
__device__ __forceinline__ void swiglu_each(float (&v)[N], const float (&u)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const F2 z(v[i], v[i + 1]);
    (z * sigmoid2(z) * F2(u[i], u[i + 1])).get(v[i], v[i + 1]);
  }
}

// d act / d z
template <int ACT>
__device__ __forceinline__ F2 act_slope2(F2 z) {
  if (ACT == kActRelu) {
    float x, y;
    z.get(x, y);  // (a NaN stays one)
    return F2(x > 0.f ? 1.f : (x <= 0.f ? 0.f : x), y > 0.f ? 1.f : (y <= 0.f ? 0.f : y));
  }
  if (ACT == kActGelu) {
    F2 density;
    const F2 c = normal_cdf2(z, &density);
    return fma2(z, density, c);
  }
  if (ACT == kActSilu) {
    const F2 s = sigmoid2(z);
    return s * fma2(z, fma2(s, F2(-1.f), F2(1.f)), F2(1.f));
  }
  return F2(1.f);
}

}  // namespace moonep
