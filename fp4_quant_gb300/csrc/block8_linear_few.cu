// y = x W^T of 8-bit operands for up to 16 tokens (glu_block8.h): bound by reading
// W once (N K bytes).  A block has 16 rows of W; its warps share the blocks of the
// sum and join in a fixed order.  The products are mma.sync (16 rows x 8 tokens x
// 32): their rate does not matter here, and their operand layout is met without
// moving data between lanes.  Of a block's 128 bytes of rows g and g + 8 (g = lane
// / 4) a lane holds 16 from 16 (lane % 4) on and 16 from 64 bytes further on (whole
// sectors in each copy); the order of a sum is free, so words 2 j and 2 j + 1 of them
// serve as the instruction's k = 4 t .. and 4 t + 16 .. of step j, with x taken the
// same way.  A block's sum is scaled and added in fp32.  Every lane copies what it
// will use itself into slots of shared memory that only it reads (cp.async), so a
// warp keeps several blocks in flight without registers or barriers.  One token of
// 7168 x 8192: 12 us, 4.8 TB/s (27 with a lane's 32 bytes next to each other, half
// sectors at a time; 25 in a tile of 32 tokens of the pairs' kernel).
#include "block8.h"
#include "block_util.cuh"

namespace gq {
namespace {

constexpr int kFewWarps8 = 4;

struct Few8P {
  const uint8_t *x, *w;
  const float *xs, *ws;
  uint16_t* y;
  int64_t ld_x, ld_w, ld_y;
  int32_t M, N, K;
};

__device__ __forceinline__ void mma_16x8x32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first n (as far as 1..16) bytes from k of a row to a slot, the rest 0.
__device__ __forceinline__ void few8_copy(uint4* slot, const uint8_t* row, int32_t k, int32_t n) {
  const uint32_t bytes = uint32_t(min(max(n, 0), 16));
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(uint32_t(__cvta_generic_to_shared(slot))),
               "l"(bytes ? row + k : row), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void few8_copy(float* slot, const float* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(uint32_t(__cvta_generic_to_shared(slot))), "l"(from) : "memory");
}

// TT: groups of eight tokens; DEEP: slots, one more than the blocks in flight.  A
// lane's slot: W's four pieces, x's two per group, and the scales: W's and of two
// tokens per group.
template <int TT>
constexpr int kSlot8 = 4 + 2 * TT + (2 * TT + 1 + 3) / 4;
template <int TT, int DEEP>
constexpr int few8_smem() {
  const int ring = kFewWarps8 * DEEP * kSlot8<TT> * 32 * 16, sums = kFewWarps8 * 16 * (8 * TT + 1) * 4;
  return ring > sums ? ring : sums;
}

template <int TT, int DEEP>
__global__ void __launch_bounds__(kFewWarps8 * 32) few8_kernel(const __grid_constant__ Few8P p) {
  extern __shared__ __align__(16) uint4 ring[];  // [warps][DEEP][kSlot8][32], then the sums
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int32_t n0 = blockIdx.x * 16;
  // rows past N are read as the last one and not stored
  const uint8_t* w0 = p.w + int64_t(min(n0 + g, p.N - 1)) * p.ld_w;
  const uint8_t* w1 = p.w + int64_t(min(n0 + g + 8, p.N - 1)) * p.ld_w;
  float c[TT][4] = {};
  // this warp's blocks of the sum
  const int32_t blocks = (p.K + kBlock8 - 1) / kBlock8, s0 = blocks * warp / kFewWarps8, s1 = blocks * (warp + 1) / kFewWarps8;
  const float* ws = p.ws + int64_t(n0 / kBlock8) * blocks;  // 16 rows of W never cross one of its blocks
  uint4* mine = ring + warp * DEEP * kSlot8<TT> * 32 + lane;
  // what belongs to tokens past M is never copied
#pragma unroll
  for (int i = 0; i < DEEP; ++i)
#pragma unroll
    for (int j = 4; j < kSlot8<TT>; ++j) mine[(i * kSlot8<TT> + j) * 32] = make_uint4(0, 0, 0, 0);
  after_previous();
  auto copy = [&](int32_t s, int slot) {
    if (s < s1) {
      const int32_t k = s * kBlock8 + 16 * t, left = p.K - k;
      uint4* q = mine + slot * kSlot8<TT> * 32;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        few8_copy(q + i * 32, w0, k + 64 * i, left - 64 * i);
        few8_copy(q + (2 + i) * 32, w1, k + 64 * i, left - 64 * i);
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          const int32_t m = 8 * j + g;
          if (m < p.M) few8_copy(q + (4 + 2 * j + i) * 32, p.x + int64_t(m) * p.ld_x, k + 64 * i, left - 64 * i);
        }
      }
      few8_copy(reinterpret_cast<float*>(q + (4 + 2 * TT) * 32), ws + s);
#pragma unroll
      for (int i = 0; i < 2 * TT; ++i) {
        const int32_t m = 8 * (i / 2) + 2 * t + (i & 1);
        if (m < p.M) few8_copy(reinterpret_cast<float*>(q + (4 + 2 * TT + (1 + i) / 4) * 32) + (1 + i) % 4, p.xs + int64_t(s) * p.M + m);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < DEEP - 1; ++i) copy(s0 + i, i);
  int slot = 0;
  for (int32_t s = s0; s < s1; ++s) {
    asm volatile("cp.async.wait_group %0;" ::"n"(DEEP - 2) : "memory");
    const uint4* q = mine + slot * kSlot8<TT> * 32;
    const uint4 a0 = q[0], a1 = q[32], b0 = q[64], b1 = q[96];
    float scale[4 * ((2 * TT + 1 + 3) / 4)];
#pragma unroll
    for (int i = 0; i < (2 * TT + 1 + 3) / 4; ++i) {
      const uint4 v = q[(4 + 2 * TT + i) * 32];
      scale[4 * i] = __uint_as_float(v.x), scale[4 * i + 1] = __uint_as_float(v.y);
      scale[4 * i + 2] = __uint_as_float(v.z), scale[4 * i + 3] = __uint_as_float(v.w);
    }
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      const uint4 v0 = q[(4 + 2 * j) * 32], v1 = q[(5 + 2 * j) * 32];
      float d[4] = {};
      mma_16x8x32(d, a0.x, b0.x, a0.y, b0.y, v0.x, v0.y);
      mma_16x8x32(d, a0.z, b0.z, a0.w, b0.w, v0.z, v0.w);
      mma_16x8x32(d, a1.x, b1.x, a1.y, b1.y, v1.x, v1.y);
      mma_16x8x32(d, a1.z, b1.z, a1.w, b1.w, v1.z, v1.w);
#pragma unroll
      for (int i = 0; i < 4; ++i) c[j][i] = fmaf(d[i], scale[0] * scale[1 + 2 * j + (i & 1)], c[j][i]);
    }
    // the slot read in the step before this one takes the next copy
    copy(s + DEEP - 1, slot == 0 ? DEEP - 1 : slot - 1);
    if (++slot == DEEP) slot = 0;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  float(*sums)[16][8 * TT + 1] = reinterpret_cast<float(*)[16][8 * TT + 1]>(ring);
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int tok = 8 * j + 2 * t;
    sums[warp][g][tok] = c[j][0];
    sums[warp][g][tok + 1] = c[j][1];
    sums[warp][g + 8][tok] = c[j][2];
    sums[warp][g + 8][tok + 1] = c[j][3];
  }
  __syncthreads();
  for (int q = threadIdx.x; q < 16 * p.M; q += kFewWarps8 * 32) {
    const int r = q & 15, m = q >> 4;
    const int32_t n = n0 + r;
    if (n >= p.N) continue;
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kFewWarps8; ++i) v += sums[i][r][m];
    p.y[m * p.ld_y + n] = bits_of_bf16(v);
  }
}

template <int TT, int DEEP>
cudaError_t launch_few8_d(const Few8P& p, cudaStream_t s) {
  constexpr int smem = few8_smem<TT, DEEP>();
  auto kern = few8_kernel<TT, DEEP>;
  static SmemLimit limit;
  const cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, unsigned((p.N + 15) / 16), kFewWarps8 * 32, smem, s, p, true);
}

// Slots by how many blocks share an SM: what is in flight per SM stays about the
// same, and all blocks are there at once up to three per SM.
template <int TT>
cudaError_t launch_few8_t(const Few8P& p, cudaStream_t s) {
  const int blocks = (p.N + 15) / 16;
  if (blocks <= 152) return launch_few8_d<TT, TT == 1 ? 14 : 10>(p, s);
  if (blocks <= 304) return launch_few8_d<TT, TT == 1 ? 7 : 5>(p, s);
  return launch_few8_d<TT, TT == 1 ? 5 : 3>(p, s);
}

}  // namespace

bool linear8_few(const glu_block8_linear_args& a) { return a.E == 0 && a.grad == 0 && a.M <= 16; }

cudaError_t launch_linear8_few(const glu_block8_linear_args& a, cudaStream_t s) {
  Few8P p;
  p.x = static_cast<const uint8_t*>(a.xq);
  p.w = static_cast<const uint8_t*>(a.wq);
  p.xs = a.xs;
  p.ws = a.ws;
  p.y = static_cast<uint16_t*>(a.y);
  p.ld_x = a.ld_x;
  p.ld_w = a.ld_w;
  p.ld_y = a.ld_y;
  p.M = int32_t(a.M);
  p.N = int32_t(a.N);
  p.K = int32_t(a.K);
  return p.M <= 8 ? launch_few8_t<1>(p, s) : launch_few8_t<2>(p, s);
}

}  // namespace gq
