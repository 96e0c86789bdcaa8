// fq_epilogue.cuh -- activations of the matrix product's epilogue, in fp32.
//
// All three smooth ones are y times a value in [0, 1] whose relative error counts where it is small: the logistic
// function of -|t| comes from exp(-|t|), never from 1 minus something, and gelu's normal distribution function is erfc of
// the other sign (1 + erf loses all its bits at y = -5). ex2.approx and rcp.approx (2 ulp) and erfcf (4 ulp) are 2^-19
// of the value at worst, with the rounding of the exponent, 256 times less than half a step of fp16.
#pragma once

#include "fq.h"
#include "fq_device.cuh"

namespace fq {

// y / (1 + exp(-t))
__device__ __forceinline__ float times_logistic(float y, float t) {
  float e, r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(-fabsf(t) * 1.44269504088896341f));
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return y * (t < 0.f ? e : 1.f) * r;
}

__device__ __forceinline__ float activate(int act, float y) {
  switch (act) {
    case FQ_ACT_RELU: return y > 0.f || y != y ? y : 0.f;  // a NaN stays one
    case FQ_ACT_GELU: return 0.5f * y * erfcf(y * -0.707106781186547524f);
    case FQ_ACT_GELU_TANH: return times_logistic(y, 1.59576912160573071f * fmaf(0.044715f * y * y, y, y));
    case FQ_ACT_SILU: return times_logistic(y, y);
    default: return y;
  }
}

}  // namespace fq
