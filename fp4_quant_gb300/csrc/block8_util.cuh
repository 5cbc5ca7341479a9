// Values to E4M3 codes with a scale per block, and back (glu_block8.h).
#pragma once

#include "block8.h"
#include "block_util.cuh"

namespace gq {

constexpr float kTop8 = 448.0f;               // the largest E4M3 value
constexpr float kLeast8 = 0x1p-100f;          // a block's maximum counts as this at least

// 1 / x to 2^-23; x and the result are not below 2^-126.
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// What a block's codes are made with and its scale; all NaN where it holds a NaN or
// an infinity, which makes its codes NaN too.  s is a / 448 rounded once: the product
// with the rounded 1 / 448, corrected by its remainder (Markstein, 1990).  r is 448 / a,
// the reciprocal of s corrected in the same way: rounded once (lo is 0), or, EXACT, in
// two parts that are within 2^-45 of it together, r rounded down and what that leaves,
// which is never negative (so that a zero keeps its sign).  All is in range for all a.
// Once per block, by the lane that has its maximum.
struct Fit8 {
  float r, lo, s;
};
template <bool EXACT>
__device__ __forceinline__ Fit8 fit8(float amax) {
  constexpr float kInv = 1.0f / kTop8;
  const float a = amax <= 3.402823466e38f ? fmaxf(amax, kLeast8) : __uint_as_float(0x7FC00000u), q = a * kInv;
  Fit8 f;
  f.s = fmaf(fmaf(-q, kTop8, a), kInv, q);
  const float y = rcp_fast(f.s), rest = fmaf(-y, a, kTop8), step = y * kInv;
  f.r = EXACT ? __fmaf_rd(rest, step, y) : fmaf(rest, step, y);
  f.lo = EXACT ? fmaxf(fmaf(-f.r, a, kTop8), 0.0f) * step : 0.0f;
  return f;
}

__device__ __forceinline__ uint32_t e4m3x2_of(float2 v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(v.y), "f"(v.x));
  return r;
}

// Codes of values of a block whose maximum is a, by their quotients 448 v / a rounded
// to fp32.  With both parts of 448 / a they are rounded once (v r + v lo is within
// 2^-45 of them before that), and one that is a midpoint of two codes stays one.  A
// quotient of bf16 values is 2^-13 (relative) away from every other midpoint at least:
// with 8-bit integers m, a' and an odd one of 5 bits t, |7 m 2^x - t a'| is 1 at
// least, and t a' < 2^13; one of products of two bf16 is 2^-21 away in the same way.
// So either gets the exact quotient's code.  Values that are rounded themselves, by
// 2^-24 at least, are multiplied with 448 / a rounded to one number, which adds a
// rounding of 2^-24 and no more (in two parts: the kept rows of 32768 x 2048 46 us
// instead of 41, the quantised backward of 32768 x 1024 94 instead of 86, cold).
__device__ __forceinline__ uint2 codes8(const F8& v, const float2 (&r)[4], const float2 (&lo)[4]) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = e4m3x2_of(fma_2(v.v[i], r[i], mul_2(v.v[i], lo[i])));
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}
__device__ __forceinline__ uint2 codes8(const F8& v, const float2 (&r)[4]) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = e4m3x2_of(mul_2(v.v[i], r[i]));
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}
__device__ __forceinline__ uint2 codes8(const F8& v, float r, float lo) {
  const float2 q[4] = {both(r), both(r), both(r), both(r)}, l[4] = {both(lo), both(lo), both(lo), both(lo)};
  return codes8(v, q, l);
}
__device__ __forceinline__ uint2 codes8(const F8& v, float r) {
  const float2 q[4] = {both(r), both(r), both(r), both(r)};
  return codes8(v, q);
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

// The first n of 16 bytes to shared memory (both on 16 bytes), the rest zeros; or a
// word, or zero.
__device__ __forceinline__ void copy16(void* dst, const void* src, uint32_t n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src), "r"(there ? 4u : 0u)
               : "memory");
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// |max| of eight values
__device__ __forceinline__ float amax8(const F8& f) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = max_nan(fabsf(f.v[i].x), fabsf(f.v[i].y));
  return max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3]));
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
// N values per lane (a power of two up to 16): lane l of the 16 gets the maximum
// over them of value l % N.  Halves, quarters, ... swap what the others keep, so
// that it takes N - 1 exchanges and one for each halving that is left.
template <int N>
__device__ __forceinline__ float scatter_max(float (&v)[N], int lane) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float got = __shfl_xor_sync(0xFFFFFFFFu, up ? v[i] : v[i + o], o);
      v[i] = max_nan(up ? v[i + o] : v[i], got);
    }
  }
#pragma unroll
  for (int o = N; o < 16; o <<= 1) v[0] = max_nan(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], o));
  return v[0];
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
  auto first = [&](int32_t e) { return min(max(offsets[e], 0), M) / kBlock8 + e; };
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
  const int32_t begin = min(max(offsets[at], 0), M), end = at < E ? min(max(offsets[at + 1], begin), M) : M;
  const int64_t r0 = begin + int64_t(tile - (begin / kBlock8 + at)) * kBlock8;
  t.r0 = int32_t(min(max(r0, int64_t(begin)), int64_t(end)));
  t.r1 = min(end, t.r0 + kBlock8);
  t.cols = at < E;
  return t;
}

}  // namespace gq
