// Matrices as E4M3 codes with a scale per block of 128 (glu_block8.h): rows
// (1 x 128), columns (128 x 1) and weights (128 x 128).  Bound by HBM: a block of
// 256 threads takes a tile of 128 x 128 values, reads it once, 16 bytes a lane,
// and keeps it in registers while the maxima of its rows (16 lanes each) and of
// its columns (through shared memory) are found.
#include "block8_util.cuh"

namespace gq {
namespace {

constexpr int kQuantWarps = 8, kRowsPerLane = 8;

struct QuantP {
  const uint16_t* x;
  const uint8_t* xq;
  const float* xs;
  const int32_t* offsets;
  uint8_t *q, *qc;
  float *s, *sc;
  int64_t ld_x, ld_xq, ld_q, ld_qc;
  int32_t M, K, E, k_tiles, col_blocks;
};

// Fits of a tile's columns, from the maxima that each warp found of its rows.
struct ColFits {
  float part[kQuantWarps][kBlock8];
  float r[kBlock8];
};

// A warp has rows 16 w .. 16 w + 15 of the tile: its lower half-warp the first
// eight, the upper one the others, a lane eight columns of each.
template <bool KEPT, bool ROWS, bool COLS>
__global__ void __launch_bounds__(kQuantWarps * 32, 4) quant8_kernel(const __grid_constant__ QuantP p) {
  __shared__ ColFits fits;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c8 = lane & 15;
  const int32_t tile = blockIdx.x / p.k_tiles, kt = blockIdx.x - tile * p.k_tiles;
  after_previous();
  const RowTile t = row_tile(p.offsets, p.E, p.M, tile);
  const bool cols = COLS && tile < p.col_blocks;
  const int32_t k = kt * kBlock8 + c8 * 8, left = p.K - k;  // of the row from this lane's columns on
  const int32_t row0 = warp * 16 + (lane >> 4) * kRowsPerLane, rows = t.r1 - t.r0 - row0;
  uint4 w[kRowsPerLane];     // bf16
  uint2 c[kRowsPerLane];     // KEPT: codes and scales
  float cs[kRowsPerLane];
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i) {
    w[i] = make_uint4(0, 0, 0, 0);
    c[i] = make_uint2(0, 0);
    cs[i] = 0.0f;
    if (i < rows && left > 0 && (ROWS || t.cols)) {
      const int64_t m = t.r0 + row0 + i;
      if (KEPT) {
        c[i] = bytes8(p.xq + m * p.ld_xq + k, left);
        cs[i] = __ldg(p.xs + int64_t(kt) * p.M + m);
      } else {
        w[i] = raw8(p.x + m * p.ld_x + k, left);
      }
    }
  }
  auto value = [&](int i) {
    if (!KEPT) return pairs(w[i]);
    F8 v = values8(c[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) v.v[j] = mul_2(v.v[j], both(cs[i]));
    return v;
  };
  if (ROWS) {
    // two rows' maxima share the exchanges; lane i of a half then fits row i
    float mine = 0.0f;
#pragma unroll
    for (int i = 0; i < kRowsPerLane; i += 2) {
      const uint32_t a = amax_bits(w[i]), b = amax_bits(w[i + 1]);
      const uint32_t m = row_max2(__vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632)));
      if (c8 == i) mine = __uint_as_float(m << 16);
      if (c8 == i + 1) mine = __uint_as_float(m & 0xFFFF0000u);
    }
    const Fit8 f = fit8(mine);
    if (c8 < kRowsPerLane && c8 < rows) p.s[int64_t(kt) * p.M + t.r0 + row0 + c8] = f.s;
#pragma unroll
    for (int i = 0; i < kRowsPerLane; ++i) {
      const float r = __shfl_sync(0xFFFFFFFFu, f.r, i, 16);
      if (i < rows && left > 0) put_bytes8(p.q + int64_t(t.r0 + row0 + i) * p.ld_q + k, left, codes8<true>(pairs(w[i]), r));
    }
  }
  if (!cols) return;
  if (!t.cols) {  // rows of no expert: their blocks are zeros
#pragma unroll
    for (int i = 0; i < kRowsPerLane; ++i) w[i] = make_uint4(0, 0, 0, 0), c[i] = make_uint2(0, 0);
  }
  float m[8];
  if (KEPT) {
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < kRowsPerLane; ++i) {
      const F8 v = value(i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m[2 * j] = max_nan(m[2 * j], fabsf(v.v[j].x));
        m[2 * j + 1] = max_nan(m[2 * j + 1], fabsf(v.v[j].y));
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = max_nan(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], 16));
  } else {
    uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kRowsPerLane; ++i) {
      u[0] = __vmaxu2(u[0], w[i].x & 0x7FFF7FFFu);
      u[1] = __vmaxu2(u[1], w[i].y & 0x7FFF7FFFu);
      u[2] = __vmaxu2(u[2], w[i].z & 0x7FFF7FFFu);
      u[3] = __vmaxu2(u[3], w[i].w & 0x7FFF7FFFu);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = __vmaxu2(u[j], __shfl_xor_sync(0xFFFFFFFFu, u[j], 16));
      m[2 * j] = __uint_as_float(u[j] << 16);
      m[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
    }
  }
  if (lane < 16) {
    float4* o = reinterpret_cast<float4*>(&fits.part[warp][c8 * 8]);
    o[0] = make_float4(m[0], m[1], m[2], m[3]);
    o[1] = make_float4(m[4], m[5], m[6], m[7]);
  }
  __syncthreads();
  if (threadIdx.x < kBlock8) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < kQuantWarps; ++i) a = max_nan(a, fits.part[i][threadIdx.x]);
    const Fit8 f = fit8(a);
    fits.r[threadIdx.x] = f.r;
    if (kt * kBlock8 + int32_t(threadIdx.x) < p.K) p.sc[int64_t(tile) * p.K + kt * kBlock8 + threadIdx.x] = f.s;
  }
  __syncthreads();
  float2 r[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = *reinterpret_cast<const float2*>(&fits.r[c8 * 8 + 2 * j]);
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i) {
    if (left > 0) put_bytes8(p.qc + (int64_t(tile) * kBlock8 + row0 + i) * p.ld_qc + k, left, codes8<!KEPT>(value(i), r));
  }
}

struct WeightP {
  const uint16_t* w;
  uint8_t* q;
  float* s;
  int64_t ld_w, stride_w, ld_q, stride_q;
  int32_t N, K, n_tiles, k_tiles;
};

__global__ void __launch_bounds__(kQuantWarps * 32, 4) weight8_kernel(const __grid_constant__ WeightP p) {
  __shared__ float part[kQuantWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c8 = lane & 15;
  const int32_t rt = blockIdx.x / p.k_tiles, kt = blockIdx.x - rt * p.k_tiles, e = rt / p.n_tiles, nt = rt - e * p.n_tiles;
  const int32_t k = kt * kBlock8 + c8 * 8, left = p.K - k;
  const int32_t row0 = nt * kBlock8 + warp * 16 + (lane >> 4) * kRowsPerLane, rows = p.N - row0;
  const uint16_t* src = p.w + e * p.stride_w + int64_t(row0) * p.ld_w + k;
  uint4 w[kRowsPerLane];
  uint32_t u = 0;
  after_previous();
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i) w[i] = i < rows && left > 0 ? raw8(src + i * p.ld_w, left) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i) u = __vmaxu2(u, amax_bits(w[i]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) u = __vmaxu2(u, __shfl_xor_sync(0xFFFFFFFFu, u, o));
  if (lane == 0) part[warp] = top_half(u);
  __syncthreads();
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < kQuantWarps; ++i) a = max_nan(a, part[i]);
  const Fit8 f = fit8(a);
  if (threadIdx.x == 0) p.s[int64_t(rt) * p.k_tiles + kt] = f.s;
  uint8_t* dst = p.q + e * p.stride_q + int64_t(row0) * p.ld_q + k;
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i)
    if (i < rows && left > 0) put_bytes8(dst + i * p.ld_q, left, codes8<true>(pairs(w[i]), f.r));
}

}  // namespace

cudaError_t launch_quant8(const glu_block8_quant_args& a, cudaStream_t s) {
  QuantP p;
  p.x = static_cast<const uint16_t*>(a.x);
  p.xq = static_cast<const uint8_t*>(a.xq);
  p.xs = a.xs;
  p.offsets = a.E > 0 ? a.offsets : nullptr;
  p.q = static_cast<uint8_t*>(a.q);
  p.qc = static_cast<uint8_t*>(a.qc);
  p.s = a.s;
  p.sc = a.sc;
  p.ld_x = a.ld_x;
  p.ld_xq = a.ld_xq;
  p.ld_q = a.ld_q;
  p.ld_qc = a.ld_qc;
  p.M = int32_t(a.M);
  p.K = int32_t(a.K);
  p.E = a.E;
  p.k_tiles = int32_t(blocks8(a.K));
  p.col_blocks = int32_t(col_blocks8(a.M, a.E));
  // by expert the rows behind the last one take up to one tile more (only the row form has them)
  const int64_t tiles = p.col_blocks + (a.E > 0 && a.q ? 1 : 0);
  auto kern = a.x == nullptr ? quant8_kernel<true, false, true>
              : a.qc == nullptr ? quant8_kernel<false, true, false>
              : a.q == nullptr ? quant8_kernel<false, false, true>
                               : quant8_kernel<false, true, true>;
  return launch_kernel(kern, unsigned(tiles * p.k_tiles), kQuantWarps * 32, 0, s, p, true);
}

cudaError_t launch_quant8_weight(const glu_block8_quant_weight_args& a, cudaStream_t s) {
  WeightP p;
  p.w = static_cast<const uint16_t*>(a.w);
  p.q = static_cast<uint8_t*>(a.q);
  p.s = a.s;
  p.ld_w = a.ld_w;
  p.stride_w = a.stride_w;
  p.ld_q = a.ld_q;
  p.stride_q = a.stride_q;
  p.N = int32_t(a.N);
  p.K = int32_t(a.K);
  p.n_tiles = int32_t(blocks8(a.N));
  p.k_tiles = int32_t(blocks8(a.K));
  const int64_t tiles = int64_t(a.E > 0 ? a.E : 1) * p.n_tiles * p.k_tiles;
  return launch_kernel(weight8_kernel, unsigned(tiles), kQuantWarps * 32, 0, s, p, true);
}

}  // namespace gq
