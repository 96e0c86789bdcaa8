// fq_epilogue.cuh -- activations of the matrix product's epilogue, in fp32, four values at a time.
//
// The smooth ones are y times a value in [0, 1] whose relative error counts where it is small, so none of them is 1 minus
// something there: the logistic function of -|t| is e / (1 + e) with e = exp(-|t|), and gelu's distribution function is
// erfc(x) / 2 of x = |y| / sqrt(2) on its falling side. What bounds them in the product's epilogue is the unit for
// reciprocals and exponentials (8 clocks for a warp, an FMA 1), so four values share a reciprocal, that of the product of
// their denominators: those are in [1, 2] (logistic) and [1, 7.4] (erfc), and a value that is NaN is kept out of it.
#pragma once

#include "fq.h"
#include "fq_device.cuh"

namespace fq {

__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// 1 / d of four positive numbers whose product is far inside fp32's range.
__device__ __forceinline__ void reciprocals(const float (&d)[4], float (&r)[4]) {
  const float a = d[0] * d[1], b = d[2] * d[3];
  float s;
  asm("rcp.approx.f32 %0, %1;" : "=f"(s) : "f"(a * b));
  const float ra = s * b, rb = s * a;
  r[0] = ra * d[1];
  r[1] = ra * d[0];
  r[2] = rb * d[3];
  r[3] = rb * d[2];
}

// y / (1 + exp(-t))
__device__ __forceinline__ void times_logistic(float (&y)[4], const float (&t)[4]) {
  float e[4], d[4], r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e[i] = fmaxf(exp2_approx(fabsf(t[i]) * -1.44269504088896341f), 0.f);  // 0 for a NaN, which y is then too
    d[i] = 1.f + e[i];
  }
  reciprocals(d, r);
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] *= (t[i] < 0.f ? e[i] : 1.f) * r[i];
}

// y * erfc(-y / sqrt(2)) / 2. erfc(x) / 2 = t * 2^(q(t) - x^2 log2 e) with t = 1 / (1 + 0.4 x) and a polynomial q, fitted to
// log2(erfc(x) exp(x^2) / (2 t)) on 0 <= x <= 12 by least squares whose weights follow the largest errors: 2^-23.4 of the
// value, and in fp32 2^-20 up to x = 3 (the rounding of x^2; 2^-17 at x = 9).
__device__ __forceinline__ void times_normal(float (&y)[4]) {
  float x[4], d[4], t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = fminf(fabsf(y[i]) * 0.707106781186547524f, 16.f);  // 16 for a NaN; erfc is 0 there
    d[i] = fmaf(0.4f, x[i], 1.f);
  }
  reciprocals(d, t);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float q = -0.30157715f;
    q = fmaf(q, t[i], 1.3452829f);
    q = fmaf(q, t[i], -2.1683304f);
    q = fmaf(q, t[i], 1.4709361f);
    q = fmaf(q, t[i], -0.66122967f);
    q = fmaf(q, t[i], 0.4430461f);
    q = fmaf(q, t[i], 0.5741099f);
    q = fmaf(q, t[i], 1.4455438f);
    q = fmaf(q, t[i], -3.1477816f);
    const float low = t[i] * exp2_approx(fmaf(x[i] * x[i], -1.44269504088896341f, q));
    y[i] *= y[i] < 0.f ? low : 1.f - low;
  }
}

template <int kAct>
__device__ __forceinline__ void activate4(float (&y)[4]) {
  if constexpr (kAct == FQ_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = y[i] <= 0.f ? 0.f : y[i];  // a NaN stays one
  } else if constexpr (kAct == FQ_ACT_GELU) {
    times_normal(y);
  } else if constexpr (kAct == FQ_ACT_GELU_TANH) {
    float t[4];  // (1 + tanh(s)) / 2 is the logistic function of 2 s
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = 1.59576912160573071f * fmaf(0.044715f * y[i] * y[i], y[i], y[i]);
    times_logistic(y, t);
  } else if constexpr (kAct == FQ_ACT_SILU) {
    const float t[4] = {y[0], y[1], y[2], y[3]};
    times_logistic(y, t);
  }
}

__device__ __forceinline__ void activate4(int act, float (&y)[4]) {
  switch (act) {
    case FQ_ACT_RELU: activate4<FQ_ACT_RELU>(y); break;
    case FQ_ACT_GELU: activate4<FQ_ACT_GELU>(y); break;
    case FQ_ACT_GELU_TANH: activate4<FQ_ACT_GELU_TANH>(y); break;
    case FQ_ACT_SILU: activate4<FQ_ACT_SILU>(y); break;
    default: break;
  }
}

}  // namespace fq
