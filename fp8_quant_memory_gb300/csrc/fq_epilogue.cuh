// fq_epilogue.cuh -- activations of the matrix product's epilogue, in fp32, two values at a time.
//
// The smooth ones are y times a value in [0, 1] whose relative error counts where it is small, so none of them is 1 minus
// something there: the logistic function of t is 1 / (1 + exp(-t)), and gelu's distribution function is erfc(x) / 2 of
// x = |y| / sqrt(2) on its falling side. In the product's epilogue they are bound by instructions and by the unit for
// reciprocals and exponentials (8 clocks for a warp, an FMA 1): pairs take one instruction where there is one for two, and
// share a reciprocal, that of the product of their denominators. Those are kept below 2^62 and above 0, so that the product
// is inside fp32's range: a logistic function below 2^-62 is 2^-62, and one of a NaN is a number (y is the NaN). y itself
// is not taken below where that begins, so that what is left there is at most 1e-17 of size however large y is.
#pragma once

#include "fq.h"
#include "fq_device.cuh"

namespace fq {

__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// (1 / d.x, 1 / d.y) of two positive numbers whose product is inside fp32's range.
__device__ __forceinline__ float2 reciprocals(float2 d) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d.x * d.y));
  return mul2(splat2(r), make_float2(d.y, d.x));
}

// The larger of the two, or NaN if y is.
__device__ __forceinline__ float at_least(float y, float least) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(y), "f"(least));
  return r;
}

// y / (1 + 2^u); u is above 62 below y = least
__device__ __forceinline__ float2 over_one_plus(float2 y, float2 u, float least) {
  const float2 e = make_float2(exp2_approx(fminf(u.x, 62.f)), exp2_approx(fminf(u.y, 62.f)));
  return mul2(make_float2(at_least(y.x, least), at_least(y.y, least)), reciprocals(add2(e, splat2(1.f))));
}

// y * erfc(-y / sqrt(2)) / 2. erfc(x) / 2 = t * 2^(q(t) - x^2 log2 e) with t = 1 / (1 + 0.4 x) and a polynomial q, fitted to
// log2(erfc(x) exp(x^2) / (2 t)) on 0 <= x <= 12 by least squares whose weights follow the largest errors: 2^-23.4 of the
// value, and in fp32 2^-20 up to x = 3 (the rounding of x^2; 2^-17 at x = 9).
__device__ __forceinline__ float2 times_normal(float2 y) {
  const float2 x = make_float2(fminf(fabsf(y.x) * 0.707106781186547524f, 16.f), fminf(fabsf(y.y) * 0.707106781186547524f, 16.f));
  const float2 t = reciprocals(fma2(splat2(0.4f), x, splat2(1.f)));
  float2 q = splat2(-0.30157715f);
  q = fma2(q, t, splat2(1.3452829f));
  q = fma2(q, t, splat2(-2.1683304f));
  q = fma2(q, t, splat2(1.4709361f));
  q = fma2(q, t, splat2(-0.66122967f));
  q = fma2(q, t, splat2(0.4430461f));
  q = fma2(q, t, splat2(0.5741099f));
  q = fma2(q, t, splat2(1.4455438f));
  q = fma2(q, t, splat2(-3.1477816f));
  const float2 u = fma2(mul2(x, x), splat2(-1.44269504088896341f), q);
  const float2 low = mul2(t, make_float2(exp2_approx(u.x), exp2_approx(u.y)));
  return mul2(y, make_float2(y.x < 0.f ? low.x : 1.f - low.x, y.y < 0.f ? low.y : 1.f - low.y));
}

template <int kAct>
__device__ __forceinline__ float2 activate2(float2 y) {
  if constexpr (kAct == FQ_ACT_RELU) {
    return make_float2(y.x <= 0.f ? 0.f : y.x, y.y <= 0.f ? 0.f : y.y);  // a NaN stays one
  } else if constexpr (kAct == FQ_ACT_GELU) {
    return times_normal(y);
  } else if constexpr (kAct == FQ_ACT_GELU_TANH) {
    // (1 + tanh(s)) / 2 is the logistic function of 2 s, s = sqrt(2 / pi) (y + 0.044715 y^3); in base 2
    const float2 f = fma2(mul2(y, y), splat2(-0.102943240f), splat2(-2.30220819f));
    return over_one_plus(y, mul2(y, f), -8.f);
  } else if constexpr (kAct == FQ_ACT_SILU) {
    return over_one_plus(y, mul2(y, splat2(-1.44269504088896341f)), -43.f);
  } else {
    return y;
  }
}

template <int kAct, int N>
__device__ __forceinline__ void activate_pairs(float2 (&y)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = activate2<kAct>(y[i]);
}

template <int N>
__device__ __forceinline__ void activate_pairs(int act, float2 (&y)[N]) {
  switch (act) {
    case FQ_ACT_RELU: activate_pairs<FQ_ACT_RELU>(y); break;
    case FQ_ACT_GELU: activate_pairs<FQ_ACT_GELU>(y); break;
    case FQ_ACT_GELU_TANH: activate_pairs<FQ_ACT_GELU_TANH>(y); break;
    case FQ_ACT_SILU: activate_pairs<FQ_ACT_SILU>(y); break;
    default: break;
  }
}

}  // namespace fq
