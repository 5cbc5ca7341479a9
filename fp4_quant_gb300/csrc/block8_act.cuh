// The gated activation's values for the operators in 8 bits: act(z) and act'(z)
// in fp32, two at a time, from ex2.approx and rcp.approx (2^-22 and 2^-23): good to a
// few 2^-23, and to |t| 2^-24 more where they go as e^-|t| (the exponent t log2 e is
// rounded once; the tanh GELU's t is a polynomial of five roundings more).  The
// blocks' codes have four bits, and it is their borders that an error crosses: with the
// exponent's rounding made up for and the reciprocal corrected, 177 instead of 182 codes
// of h in 1e8 differ from 64 bits (SiLU of N(0, 1) gates; fp32 functions and divisions
// 167), for 47 instead of 44 us (GELU 53 instead of 45, the quantised backward 95
// instead of 86, cold).
#pragma once

#include "block8_util.cuh"

namespace gq {

// 2^x and 1 / x; results and operands below 2^-126 are 0.
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 1 / (1 + 2^t)
__device__ __forceinline__ float2 sigmoid_of(float2 t) {
  const float2 e = add_2(make_float2(exp2_fast(t.x), exp2_fast(t.y)), both(1.0f));
  return make_float2(rcp_fast(e.x), rcp_fast(e.y));
}

// SiLU: s = 1 / (1 + e^-z), act = z s, act' = s + act (1 - s).
// GELU (tanh): the same s of u = 2 sqrt(2 / pi) (z + 0.044715 z^3), act = z s, act' =
// s + act (1 - s) u'.  z^2 is limited at 128^2, where s is 0 or 1 long since: u'
// stays finite, so that times 1 - s = 0 it is 0.
// Large |z| need nothing else: s is 0 or 1 exactly, and z s, 1 - s follow.
template <int ACT>
__device__ __forceinline__ void act8(float2 z, float2& a, float2& d) {
  constexpr float kLog2e = 1.4426950408889634f, kU = 1.5957691216057308f, kCubic = 0.044715f;
  if (ACT == GLU_ACT_SILU) {
    const float2 s = sigmoid_of(mul_2(z, both(-kLog2e)));
    a = mul_2(z, s);
    d = fma_2(a, fma_2(s, both(-1.0f), both(1.0f)), s);
  } else if (ACT == GLU_ACT_GELU_TANH) {
    float2 q = mul_2(z, z);
    q = make_float2(fminf(q.x, 16384.0f), fminf(q.y, 16384.0f));
    const float2 s = sigmoid_of(mul_2(z, fma_2(q, both(-kLog2e * kU * kCubic), both(-kLog2e * kU))));
    a = mul_2(z, s);
    const float2 rest = mul_2(a, fma_2(s, both(-1.0f), both(1.0f)));
    d = fma_2(rest, fma_2(q, both(kU * 3.0f * kCubic), both(kU)), s);
  } else if (ACT == GLU_ACT_RELU) {
    a = make_float2(max_nan(z.x, 0.0f), max_nan(z.y, 0.0f));
    d = make_float2(z.x <= 0.0f ? 0.0f : 1.0f, z.y <= 0.0f ? 0.0f : 1.0f);
  } else if (ACT == GLU_ACT_GELU_ERF) {
    // z and z^2 limited where the distribution function is 0 or 1
    const float2 c = make_float2(fminf(fmaxf(z.x, -128.0f), 128.0f), fminf(fmaxf(z.y, -128.0f), 128.0f));
    const float2 f = make_float2(normcdff(c.x), normcdff(c.y)), t = mul_2(mul_2(c, c), both(-0.5f * kLog2e));
    a = mul_2(z, f);
    d = fma_2(mul_2(c, both(0.3989422804014327f)), make_float2(exp2_fast(t.x), exp2_fast(t.y)), f);
  } else {
    a = z;
    d = both(1.0f);
  }
}

}  // namespace gq
