// The activations of the linear layers and their derivatives, on fp32 values
// that are rounded to bf16 next or summed in fp32.
#pragma once

#include <cuda_runtime.h>

#include "glu_quant.h"

namespace gq {

// The normal distribution function, from Abramowitz and Stegun's formula
// 7.1.26 for erf (absolute error below 1.5e-7): with v = |z| / sqrt 2 and t = 1
// / (1 + 0.3275911 v), 1 - Phi(|z|) = t (a1 + t (a2 + ...)) exp(-v^2) / 2.
__device__ __forceinline__ float normal_cdf(float z, float exp_half_sq) {
  const float t = __fdividef(1.0f, fmaf(0.3275911f * 0.70710678f, fabsf(z), 1.0f));
  float q = fmaf(1.061405429f, t, -1.453152027f);
  q = fmaf(q, t, 1.421413741f);
  q = fmaf(q, t, -0.284496736f);
  q = fmaf(q, t, 0.254829592f);
  q = 0.5f * q * t * exp_half_sq;
  return z < 0.0f ? q : 1.0f - q;
}

// act(z), for values that are rounded to bf16 next.
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == GLU_ACT_SILU) return __fdividef(z, 1.0f + __expf(-z));
  if (ACT == GLU_ACT_GELU_TANH) {
    const float u = 1.5957691216057308f * fmaf(0.044715f * z * z, z, z);  // 2 sqrt(2 / pi) (z + 0.044715 z^3)
    return __fdividef(z, 1.0f + __expf(-u));                              // z sigmoid(u) = z (1 + tanh(u / 2)) / 2
  }
  if (ACT == GLU_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
  if (ACT == GLU_ACT_GELU_ERF) return z * normal_cdf(z, __expf(-0.5f * z * z));
  return z;
}

// act'(z), |z| up to 128 or NaN: an exponential and a quotient each (the SM's
// special functions are what this kernel would wait for); 1 - s has an absolute
// error of 2^-24, which is what act' is good to.
template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
  if (ACT == GLU_ACT_SILU) {
    const float s = __fdividef(1.0f, 1.0f + __expf(-z));
    return s * fmaf(z, 1.0f - s, 1.0f);
  }
  if (ACT == GLU_ACT_GELU_TANH) {
    const float z2 = z * z;
    const float u = 1.5957691216057308f * fmaf(0.044715f * z2, z, z);
    const float du = 1.5957691216057308f * fmaf(0.134145f, z2, 1.0f);
    const float s = __fdividef(1.0f, 1.0f + __expf(-u));
    return s * fmaf(z * (1.0f - s), du, 1.0f);
  }
  if (ACT == GLU_ACT_RELU) return z <= 0.0f ? 0.0f : 1.0f;  // 1 at NaN too, as glu_act says
  if (ACT == GLU_ACT_GELU_ERF) {
    const float e = __expf(-0.5f * z * z);
    return fmaf(z * 0.3989422804014327f, e, normal_cdf(z, e));
  }
  return 1.0f;
}

// act' of two bf16.  From |z| = 128 on act' of the smooth ones is 0 or 1 in fp32,
// and z is taken as that (NaN kept): z^2 and z^3 of larger ones pass fp32's
// range, and 0 times infinity would be NaN where act' is 0 or 1 (as it is at
// infinities, the limits).  Both at once, in bf16, which holds 128: 4096 x 1462
// with SiLU takes 16.8 us, limited one by one in fp32 18.8; 16384 x 8192 99 us,
// and 91 without limits.
template <int ACT>
__device__ __forceinline__ float2 act_grad_of(uint32_t z) {
  if (ACT == GLU_ACT_SILU || ACT == GLU_ACT_GELU_TANH || ACT == GLU_ACT_GELU_ERF)
    asm("max.NaN.bf16x2 %0, %0, %1;\n\tmin.NaN.bf16x2 %0, %0, %2;" : "+r"(z) : "r"(0xC300C300u), "r"(0x43004300u));
  return make_float2(act_grad<ACT>(__uint_as_float(z << 16)), act_grad<ACT>(__uint_as_float(z & 0xFFFF0000u)));
}

}  // namespace gq
