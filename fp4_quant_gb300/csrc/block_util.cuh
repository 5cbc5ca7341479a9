// Loads and stores of eight consecutive elements as fp32, for rows whose
// width need not be a multiple of eight (rows start on 16 bytes), and the
// reductions of a warp and a block in a fixed order.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "glu_quant.h"

namespace gq {

// Launches a kernel of one parameter block; the launch's own error only.
template <typename P>
inline cudaError_t launch_kernel(void (*kern)(const P), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float bf16_of_bits(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }
__device__ __forceinline__ uint16_t bits_of_bf16(float v) { return uint16_t(bf16x2_of(v, 0.0f) & 0xFFFFu); }

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(x[i] << 16);
    v[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(bf16x2_of(v[0], v[1]), bf16x2_of(v[2], v[3]), bf16x2_of(v[4], v[5]), bf16x2_of(v[6], v[7]));
}

// Streamed data: read once, kept out of L1.
__device__ __forceinline__ uint4 ldg_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void stg_once(void* p, const uint4& v) {
  asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// The first n (1..8) bf16 of a chunk as they are; the rest is 0.
__device__ __forceinline__ uint4 raw8(const uint16_t* p, int n) {
  if (n >= 8) return ldg_once(p);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (2 * i < n ? uint32_t(p[2 * i]) : 0u) | (2 * i + 1 < n ? uint32_t(p[2 * i + 1]) << 16 : 0u);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The first n (1..8) elements of a chunk; the rest of v is 0.
__device__ __forceinline__ void load8(const uint16_t* p, int n, float (&v)[8]) {
  if (n >= 8) {
    unpack8(ldg_once(p), v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? bf16_of_bits(p[i]) : 0.0f;
  }
}
__device__ __forceinline__ void load8(const float* p, int n, float (&v)[8]) {
  if (n >= 8) {
    const uint4 a = ldg_once(p), b = ldg_once(p + 4);
    v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
  }
}
__device__ __forceinline__ void store8(uint16_t* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    stg_once(p, pack8(v));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = bits_of_bf16(v[i]);
  }
}
__device__ __forceinline__ void store8(float* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    stg_once(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
    stg_once(p + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}

// Eight elements of a vector operand (bf16 or fp32, 16-byte aligned base) from
// element c on, kept in L1; `add` is added to each.
__device__ __forceinline__ void vec8(const void* base, bool f32, int64_t c, int n, float add, float (&v)[8]) {
  if (n >= 8) {
    if (f32) {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(base) + c);
      const float4 a = __ldg(q), b = __ldg(q + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + c)), v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = i >= n ? 0.0f : f32 ? static_cast<const float*>(base)[c + i] : bf16_of_bits(static_cast<const uint16_t*>(base)[c + i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += add;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sums over the first `threads` threads of the block (whole warps; the others
// do not call) of N values each, the same bits in every thread.  `buf`
// alternates between calls (two buffers), so one barrier per call is enough:
// a buffer is written again only after the next call's barrier.
template <int N>
struct BlockSum {
  float part[2][32][N];
};
template <int N>
__device__ __forceinline__ void block_sum(BlockSum<N>& s, uint32_t& buf, int threads, float (&v)[N]) {
  const int warps = threads >> 5;
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = warp_sum(v[j]);
  if (warps == 1) {
    __syncwarp();
    return;
  }
  float(&p)[32][N] = s.part[buf & 1u];
  ++buf;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int j = 0; j < N; ++j) p[threadIdx.x >> 5][j] = v[j];
  }
  asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = 0.0f;
  for (int w = 0; w < warps; ++w) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] += p[w][j];
  }
}

}  // namespace gq
