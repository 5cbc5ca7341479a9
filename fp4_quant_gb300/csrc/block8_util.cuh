// Values to E4M3 codes with a scale per block, and back (glu_block8.h).
#pragma once

#include "block8.h"
#include "block_util.cuh"

namespace gq {

constexpr float kTop8 = 448.0f;               // the largest E4M3 value
constexpr float kLeast8 = 0x1p-100f;          // a block's maximum counts as this at least

// What a block's codes are made with: v * r rounded, unless the block holds a
// NaN or an infinity (bad: all ones in the codes' seven value bits, NaN).
struct Fit8 {
  float r, s;
  uint32_t bad;
};
__device__ __forceinline__ Fit8 fit8(float amax) {
  Fit8 f;
  const bool ok = amax <= 3.402823466e38f;
  const float a = fmaxf(amax, kLeast8);
  f.r = ok ? __fdiv_rn(kTop8, a) : 0.0f;
  f.s = ok ? __fdiv_rn(a, kTop8) : __uint_as_float(0x7FC00000u);
  f.bad = ok ? 0u : 0x7F7F7F7Fu;
  return f;
}

// For bf16 values the exact quotient 448 v / a is either the midpoint of two
// codes or 2^-13 (relative) away from it at least: with 8-bit integers m, a' and an
// odd one of 5 bits t, |7 m 2^x - t a'| is 0 or 1 at least, and t a' < 2^13.
// RN(448 / a) * v is within 2^-22 of it, so rounded to 16 significant bits it is
// on the quotient's side of every midpoint, and on the midpoint where that is.
__device__ __forceinline__ float snap8(float t) { return __uint_as_float((__float_as_uint(t) + 0x80u) & 0xFFFFFF00u); }

__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Codes of eight values, scaled by r (one for all, or pairs).  SNAP: they are bf16 values.
template <bool SNAP>
__device__ __forceinline__ uint2 codes8(const F8& v, const float2 (&r)[4]) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = mul_2(v.v[i], r[i]);
    h[i] = SNAP ? e4m3x2_of(snap8(t.x), snap8(t.y)) : e4m3x2_of(t.x, t.y);
  }
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}
template <bool SNAP>
__device__ __forceinline__ uint2 codes8(const F8& v, float r, uint32_t bad) {
  const float2 q[4] = {both(r), both(r), both(r), both(r)};
  uint2 c = codes8<SNAP>(v, q);
  c.x |= bad, c.y |= bad;
  return c;
}

// What eight codes stand for without their scale, exact in fp32.
__device__ __forceinline__ F8 values8(const uint2& c) {
  F8 f;
  const uint32_t x[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(x[i / 2] >> (16 * (i & 1)))));
    asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(f.v[i].x), "=f"(f.v[i].y) : "r"(h));
  }
  return f;
}

// The first n (1..8) bytes of a chunk (8-byte aligned), the rest 0, and back.
__device__ __forceinline__ uint2 bytes8(const uint8_t* p, int n) {
  if (n >= 8) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
  }
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) w[i / 4] |= uint32_t(p[i]) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void put_bytes8(uint8_t* p, int n, const uint2& v) {
  if (n >= 8) {
    asm volatile("st.global.cs.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(v.x), "r"(v.y) : "memory");
  } else {
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = uint8_t(w[i / 4] >> (8 * (i & 3)));
  }
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// |max| of eight values
__device__ __forceinline__ float amax8(const F8& f) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max_nan(m, max_nan(fabsf(f.v[i].x), fabsf(f.v[i].y)));
  return m;
}
// Largest bits of |v| of bf16 pairs (infinities and NaN above all others).
__device__ __forceinline__ uint32_t amax_bits(const uint4& w) {
  constexpr uint32_t k = 0x7FFF7FFFu;
  return __vmaxu2(__vmaxu2(w.x & k, w.y & k), __vmaxu2(w.z & k, w.w & k));
}
// The larger half of a pair of bf16 bits as fp32.
__device__ __forceinline__ float top_half(uint32_t w) { return __uint_as_float(max(w << 16, w & 0xFFFF0000u)); }

// Over the 16 lanes that share a row.
__device__ __forceinline__ uint32_t row_max2(uint32_t v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = __vmaxu2(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// The rows of one 128-row tile: block `tile` of the column form, and rows r0 ..
// r1 - 1 (fewer than 128 where an expert or the matrix ends; none in a block of
// no expert).  By expert there is one tile more than column blocks, and the rows
// behind the last expert take the blocks that an expert E would: those are rows
// of no column block (cols false), whose blocks are zeros.
struct RowTile {
  int32_t r0, r1;
  bool cols;
};
// By a warp; the same in every lane.  Two rounds of 32 loads find the expert.
__device__ __forceinline__ RowTile row_tile(const int32_t* offsets, int32_t E, int32_t M, int32_t tile) {
  RowTile t;
  if (offsets == nullptr) {
    t.r0 = tile * kBlock8;
    t.r1 = min(M, t.r0 + kBlock8);
    t.cols = true;
    return t;
  }
  const int lane = threadIdx.x & 31;
  auto first = [&](int32_t e) { return min(max(__ldg(offsets + e), 0), M) / kBlock8 + e; };
  // the last expert of 0 .. E (E: the rows behind the last) that begins at or before the tile
  const int32_t step = E / 32 + 1;
  int32_t e = lane * step;
  uint32_t hit = __ballot_sync(0xFFFFFFFFu, e <= E && first(min(e, E)) <= tile);
  const int32_t base = (hit ? 31 - __clz(hit) : 0) * step;
  e = base + lane;
  int32_t at = base;
  for (int32_t o = 0; o < step; o += 32) {
    hit = __ballot_sync(0xFFFFFFFFu, o + lane < step && e + o <= E && first(min(e + o, E)) <= tile);
    if (hit) at = base + o + 31 - __clz(hit);
  }
  const int32_t begin = min(max(__ldg(offsets + at), 0), M), end = at < E ? min(max(__ldg(offsets + at + 1), begin), M) : M;
  const int64_t r0 = begin + int64_t(tile - (begin / kBlock8 + at)) * kBlock8;
  t.r0 = int32_t(min(max(r0, int64_t(begin)), int64_t(end)));
  t.r1 = min(end, t.r0 + kBlock8);
  t.cols = at < E;
  return t;
}

}  // namespace gq
