// The gated activation's values for the operators in 8 bits: act(z) and act'(z)
// in fp32, good to a few 2^-23 (their blocks' scales are fp32).
#pragma once

#include "block8_util.cuh"

namespace gq {

// The smooth ones meet their limits, 0 or z and 0 or 1, before |z| = 128 in fp32;
// beyond it z^2 and z^3 would pass fp32's range, and 0 times infinity is NaN.
__device__ __forceinline__ float limit128(float z) {
  float r;
  asm("max.NaN.f32 %0, %1, 0fC3000000;\n\tmin.NaN.f32 %0, %0, 0f43000000;" : "=f"(r) : "f"(z));
  return r;
}

template <int ACT>
__device__ __forceinline__ void act8(float z, float& a, float& d) {
  if (ACT == GLU_ACT_SILU) {
    const float s = __fdividef(1.0f, 1.0f + __expf(-z)), c = limit128(z);
    a = z * s;
    d = s * fmaf(c, 1.0f - s, 1.0f);
  } else if (ACT == GLU_ACT_GELU_TANH) {
    const float c = limit128(z), c2 = c * c;
    const float u = 1.5957691216057308f * fmaf(0.044715f * c2, c, c);  // 2 sqrt(2 / pi) (z + 0.044715 z^3)
    const float s = __fdividef(1.0f, 1.0f + __expf(-u));               // (1 + tanh(u / 2)) / 2
    a = z * s;
    d = s * fmaf(c * (1.0f - s), 1.5957691216057308f * fmaf(0.134145f, c2, 1.0f), 1.0f);
  } else if (ACT == GLU_ACT_RELU) {
    a = z > 0.0f ? z : (z != z ? z : 0.0f);
    d = z <= 0.0f ? 0.0f : 1.0f;
  } else if (ACT == GLU_ACT_GELU_ERF) {
    const float c = limit128(z), f = normcdff(c);
    a = z * f;
    d = fmaf(c * 0.3989422804014327f, __expf(-0.5f * c * c), f);
  } else {
    a = z;
    d = 1.0f;
  }
}

}  // namespace gq
