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

// The larger of the two, or NaN if y is.
__device__ __forceinline__ float at_least(float y, float least) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(y), "f"(least));
  return r;
}

// d = (1 / d.x, 1 / d.y) of pairs of positive numbers whose product is inside fp32's range.
template <int N>
__device__ __forceinline__ void reciprocals(float2 (&d)[N]) {
  float r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) asm("rcp.approx.f32 %0, %1;" : "=f"(r[i]) : "f"(d[i].x * d[i].y));
#pragma unroll
  for (int i = 0; i < N; ++i) d[i] = mul2(splat2(r[i]), make_float2(d[i].y, d[i].x));
}

// y = y / (1 + 2^u); u is above 62 below y = least
template <int N>
__device__ __forceinline__ void over_one_plus(float2 (&y)[N], float2 (&u)[N], float least) {
#pragma unroll
  for (int i = 0; i < N; ++i) u[i] = make_float2(exp2_approx(fminf(u[i].x, 62.f)), exp2_approx(fminf(u[i].y, 62.f)));
#pragma unroll
  for (int i = 0; i < N; ++i) u[i] = add2(u[i], splat2(1.f));
  reciprocals(u);
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = mul2(make_float2(at_least(y[i].x, least), at_least(y[i].y, least)), u[i]);
}

// y = y * erfc(-y / sqrt(2)) / 2. erfc(x) / 2 = t * 2^(q(t) - x^2 log2 e) with t = 1 / (1 + 0.4 x) and a polynomial q, fitted
// to log2(erfc(x) exp(x^2) / (2 t)) on 0 <= x <= 12 by least squares whose weights follow the largest errors: 2^-23.4 of the
// value, and in fp32 2^-20 up to x = 3 (the rounding of x^2; 2^-17 at x = 9).
template <int N>
__device__ __forceinline__ void times_normal(float2 (&y)[N]) {
  constexpr float kQ[] = {1.3452829f, -2.1683304f, 1.4709361f, -0.66122967f, 0.4430461f, 0.5741099f, 1.4455438f, -3.1477816f};
  float2 x[N], t[N], q[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = make_float2(fminf(fabsf(y[i].x) * 0.707106781186547524f, 16.f), fminf(fabsf(y[i].y) * 0.707106781186547524f, 16.f));
    t[i] = fma2(splat2(0.4f), x[i], splat2(1.f));
    q[i] = splat2(-0.30157715f);
  }
  reciprocals(t);
#pragma unroll
  for (int k = 0; k < 8; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = fma2(q[i], t[i], splat2(kQ[k]));
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 u = fma2(mul2(x[i], x[i]), splat2(-1.44269504088896341f), q[i]);
    q[i] = make_float2(exp2_approx(u.x), exp2_approx(u.y));
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 low = mul2(t[i], q[i]);
    y[i] = mul2(y[i], make_float2(y[i].x < 0.f ? low.x : 1.f - low.x, y[i].y < 0.f ? low.y : 1.f - low.y));
  }
}

// Pairs side by side: each is a chain through two or three units, and the product has two warps to a scheduler (4096 x 8192 x
// 4096 with gelu_tanh, 16 at a time: 135 us, one after another 8 more).
template <int kAct, int N>
__device__ __forceinline__ void activate_pairs(float2 (&y)[N]) {
  if constexpr (kAct == FQ_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = make_float2(y[i].x <= 0.f ? 0.f : y[i].x, y[i].y <= 0.f ? 0.f : y[i].y);  // a NaN stays one
  } else if constexpr (kAct == FQ_ACT_GELU) {
    times_normal(y);
  } else if constexpr (kAct == FQ_ACT_GELU_TANH) {
    // (1 + tanh(s)) / 2 is the logistic function of 2 s, s = sqrt(2 / pi) (y + 0.044715 y^3); in base 2
    float2 u[N];
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = mul2(y[i], fma2(mul2(y[i], y[i]), splat2(-0.102943240f), splat2(-2.30220819f)));
    over_one_plus(y, u, -8.f);
  } else if constexpr (kAct == FQ_ACT_SILU) {
    float2 u[N];
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = mul2(y[i], splat2(-1.44269504088896341f));
    over_one_plus(y, u, -43.f);
  }
}

// The same, pair by pair, of an activation known to the launch alone: less code, which short launches fetch anew.
template <int kAct, int N>
__device__ __forceinline__ void activate_each(float2 (&y)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float2 one[1] = {y[i]};
    activate_pairs<kAct>(one);
    y[i] = one[0];
  }
}

template <int N>
__device__ __forceinline__ void activate_each(int act, float2 (&y)[N]) {
  switch (act) {
    case FQ_ACT_RELU: activate_each<FQ_ACT_RELU>(y); break;
    case FQ_ACT_GELU: activate_each<FQ_ACT_GELU>(y); break;
    case FQ_ACT_GELU_TANH: activate_each<FQ_ACT_GELU_TANH>(y); break;
    case FQ_ACT_SILU: activate_each<FQ_ACT_SILU>(y); break;
    default: break;
  }
}

}  // namespace fq
