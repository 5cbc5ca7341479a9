// Loads and stores of eight consecutive elements as fp32, for rows whose
// width need not be a multiple of eight (rows start on 16 bytes), and the
// reductions of a warp and a block in a fixed order.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "glu_quant.h"

namespace gq {

// Raises a kernel's limit of dynamic shared memory, once per device: one object
// per kernel, static where it is launched (the call costs as much as a launch).
class SmemLimit {
 public:
  cudaError_t raise(const void* kern, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kDevices && set_[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < kDevices) set_[dev].store(bytes, std::memory_order_relaxed);
    return e;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> set_[kDevices] = {};
};

// Launches a kernel of one parameter block; the launch's own error only.
// `early`: its blocks may come while the kernel before it on the stream drains;
// it then begins with after_previous(), before it touches memory.
template <typename P>
inline cudaError_t launch_kernel(void (*kern)(const P), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const P& p,
                                 bool early = false) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}
// Waits until the kernels before this one on the stream are done and what they
// wrote is there.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel's blocks may come before this one's leave (they wait for its
// end).  Only the norms let them: elsewhere blocks that wait took the place of
// ones that work (the sort of 16384 x 8 assignments and their rows 128 against
// 113 us, one token's linear layer 22.2 against 19.7 us).
__device__ __forceinline__ void next_may_come() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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

// A chunk's first n < 8 elements are moved as up to four, two and one (chunks
// start on 16 bytes).
//
// The first n (1..8) bf16 of a chunk as they are; the rest is 0.
__device__ __forceinline__ uint4 raw8(const uint16_t* p, int n) {
  if (n >= 8) return ldg_once(p);
  uint2 four = make_uint2(0u, 0u);
  uint32_t two = 0u, one = 0u;
  if (n & 4) four = *reinterpret_cast<const uint2*>(p);
  if (n & 2) two = *reinterpret_cast<const uint32_t*>(p + (n & 4));
  if (n & 1) one = p[n & 6];
  const uint32_t lo = (n & 2) ? two : one, hi = (n & 2) ? one : 0u;
  return (n & 4) ? make_uint4(four.x, four.y, lo, hi) : make_uint4(lo, hi, 0u, 0u);
}

// The first n (1..8) elements of a chunk; the rest of v is 0.
__device__ __forceinline__ void load8(const uint16_t* p, int n, float (&v)[8]) {
  unpack8(raw8(p, n), v);
}
__device__ __forceinline__ void load8(const float* p, int n, float (&v)[8]) {
  if (n >= 8) {
    const uint4 a = ldg_once(p), b = ldg_once(p + 4);
    v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
  } else {
    float4 four = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float2 two = make_float2(0.0f, 0.0f);
    float one = 0.0f;
    if (n & 4) four = *reinterpret_cast<const float4*>(p);
    if (n & 2) two = *reinterpret_cast<const float2*>(p + (n & 4));
    if (n & 1) one = p[n & 6];
    const float x = (n & 2) ? two.x : one, y = two.y, z = (n & 2) ? one : 0.0f;
    v[0] = (n & 4) ? four.x : x, v[1] = (n & 4) ? four.y : y, v[2] = (n & 4) ? four.z : z, v[3] = four.w;
    v[4] = (n & 4) ? x : 0.0f, v[5] = (n & 4) ? y : 0.0f, v[6] = (n & 4) ? z : 0.0f, v[7] = 0.0f;
  }
}
// The first n (up to 8) of eight bf16 as they are.
__device__ __forceinline__ void put8(uint16_t* p, int n, const uint4& v) {
  if (n >= 8) {
    stg_once(p, v);
  } else if (n > 0) {
    if (n & 4) *reinterpret_cast<uint2*>(p) = make_uint2(v.x, v.y);
    const uint32_t lo = (n & 4) ? v.z : v.x, hi = (n & 4) ? v.w : v.y;
    if (n & 2) *reinterpret_cast<uint32_t*>(p + (n & 4)) = lo;
    if (n & 1) p[n & 6] = uint16_t((n & 2) ? hi : lo);
  }
}
__device__ __forceinline__ void store8(uint16_t* p, int n, const float (&v)[8]) { put8(p, n, pack8(v)); }
__device__ __forceinline__ void store8(float* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    stg_once(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
    stg_once(p + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
  } else if (n > 0) {
    if (n & 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    const float x = (n & 4) ? v[4] : v[0], y = (n & 4) ? v[5] : v[1], z = (n & 4) ? v[6] : v[2];
    if (n & 2) *reinterpret_cast<float2*>(p + (n & 4)) = make_float2(x, y);
    if (n & 1) p[n & 6] = (n & 2) ? z : x;
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

// Eight values as pairs for the two-wide fp32 instructions.
struct F8 {
  float2 v[4];
};
__device__ __forceinline__ uint64_t pair_bits(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 pair_of(uint64_t r) {
  float2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
  return a;
}
__device__ __forceinline__ float2 fma_2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair_bits(a)), "l"(pair_bits(b)), "l"(pair_bits(c)));
  return pair_of(r);
}
__device__ __forceinline__ float2 mul_2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return pair_of(r);
}
__device__ __forceinline__ float2 add_2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return pair_of(r);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

__device__ __forceinline__ F8 pairs(const float (&v)[8]) {
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) f.v[i] = make_float2(v[2 * i], v[2 * i + 1]);
  return f;
}
__device__ __forceinline__ F8 zeros() {
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) f.v[i] = make_float2(0.0f, 0.0f);
  return f;
}
__device__ __forceinline__ F8 pairs(const uint4& w) {
  F8 f;
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f.v[i] = make_float2(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xFFFF0000u));
  return f;
}
__device__ __forceinline__ uint4 packed(const F8& f) {
  return make_uint4(bf16x2_of(f.v[0].x, f.v[0].y), bf16x2_of(f.v[1].x, f.v[1].y), bf16x2_of(f.v[2].x, f.v[2].y),
                    bf16x2_of(f.v[3].x, f.v[3].y));
}
// RAGGED: the width may end inside the chunk (n elements of it are stored).
template <bool RAGGED, typename T>
__device__ __forceinline__ void store8(T* p, int n, const F8& f) {
  const float v[8] = {f.v[0].x, f.v[0].y, f.v[1].x, f.v[1].y, f.v[2].x, f.v[2].y, f.v[3].x, f.v[3].y};
  store8(p, RAGGED ? n : 8, v);
}
__device__ __forceinline__ float sum2(float2 a) { return a.x + a.y; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Barrier of the block's `threads` threads (whole warps).  The warp converges
// first: an aligned barrier that its lanes reached apart (the compiler may
// place it behind either side of a branch) would count them twice.
__device__ __forceinline__ void row_barrier(int threads) {
  __syncwarp();
  asm volatile("barrier.sync 1, %0;" ::"r"(threads) : "memory");
}

// Sums over the block's `threads` threads (whole warps) of N = 1, 2 or 3 values
// each, the same bits in every thread.  `buf` alternates between calls (two
// buffers), so one barrier per call is enough: a buffer is written again only
// after the next call's barrier.  Two or three values share the exchanges inside
// a warp: halves of it first swap values, so that each half or quarter then
// sums one (5 exchanges instead of 10, 6 instead of 15).  Up to 32 warps for one
// value, up to 16 for more: those lie side by side, 16 floats each, so that a
// lane reads the float of its own number.  (As rows [N][32], read at [lane / 16]
// [lane % 16], CUDA 13.0's optimiser read every third float where such a call
// stood ahead of a loop with another.)
template <int N>
struct BlockSum {
  float part[2][N == 1 ? 32 : 16 * N];
};
__device__ __forceinline__ void block_sum(BlockSum<1>& s, uint32_t& buf, int threads, float (&v)[1]) {
  const int warps = threads >> 5, lane = threadIdx.x & 31;
  v[0] = warp_sum(v[0]);
  if (warps == 1) {
    __syncwarp();
    return;
  }
  float* q = s.part[buf & 1u];
  ++buf;
  if (lane == 0) q[threadIdx.x >> 5] = v[0];
  row_barrier(threads);
  v[0] = warp_sum(lane < warps ? q[lane] : 0.0f);
}
__device__ __forceinline__ void block_sum(BlockSum<2>& s, uint32_t& buf, int threads, float (&v)[2]) {
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  const int warps = threads >> 5, lane = threadIdx.x & 31;
  const bool hi = lane & 16;
  float x = (hi ? v[1] : v[0]) + __shfl_xor_sync(kAll, hi ? v[0] : v[1], 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(kAll, x, o);  // lanes 0-15: v[0], 16-31: v[1]
  if (warps > 1) {
    float* q = s.part[buf & 1u];
    ++buf;
    if ((lane & 15) == 0) q[lane + (threadIdx.x >> 5)] = x;
    row_barrier(threads);
    x = (lane & 15) < warps ? q[lane] : 0.0f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
  } else {
    __syncwarp();
  }
  v[0] = __shfl_sync(kAll, x, 0);
  v[1] = __shfl_sync(kAll, x, 16);
}
__device__ __forceinline__ void block_sum(BlockSum<3>& s, uint32_t& buf, int threads, float (&v)[3]) {
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  const int warps = threads >> 5, lane = threadIdx.x & 31;
  const bool hi = lane & 16, up = lane & 8;
  float a = hi ? v[2] : v[0], b = hi ? 0.0f : v[1];
  a += __shfl_xor_sync(kAll, hi ? v[0] : v[2], 16);
  b += __shfl_xor_sync(kAll, hi ? v[1] : 0.0f, 16);
  float x = (up ? b : a) + __shfl_xor_sync(kAll, up ? a : b, 8);  // lanes 0-7: v[0], 8-15: v[1], 16-23: v[2]
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
  if (warps == 1) {
#pragma unroll
    for (int j = 0; j < 3; ++j) v[j] = __shfl_sync(kAll, x, 8 * j);
    __syncwarp();
    return;
  }
  float* q = s.part[buf & 1u];
  ++buf;
  if ((lane & 7) == 0 && lane < 24) q[2 * lane + (threadIdx.x >> 5)] = x;
  row_barrier(threads);
  const bool has = (lane & 15) < warps;
  a = has ? q[lane] : 0.0f;
  b = has ? q[32 + (lane & 15)] : 0.0f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    a += __shfl_xor_sync(kAll, a, o);
    b += __shfl_xor_sync(kAll, b, o);
  }
  v[0] = __shfl_sync(kAll, a, 0);
  v[1] = __shfl_sync(kAll, a, 16);
  v[2] = b;
}

}  // namespace gq
