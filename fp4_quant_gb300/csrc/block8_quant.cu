// Matrices as E4M3 codes with a scale per block of 128 (glu_block8.h): rows
// (1 x 128), columns (128 x 1) and weights (128 x 128).
//
// Rows and columns: blocks of 256 threads walk tiles of 128 x 128 values, three per
// SM.  The next tile is on its way into shared memory while this one's maxima are
// found, of rows by 16 lanes and of columns through shared memory, and its codes
// are stored: 4096 x 7168 as rows and columns in calls of 20.9 us (119 MB, 5.7 TB/s),
// 32768 x 2048 kept rows of 64 experts as columns 35.7.  The copies are hidden (one
// block per tile with its values in registers: 24.8 and 41.9).  No unit is full: warps
// issue in 60 and 66 % of the cycles, the integer pipe works in 62 and 54 %, DRAM in 36
// and 17 %.  Five warps per scheduler are too few to fill the rest: of the 8 cycles
// between a warp's instructions it waits 1.4 and 1.1 for that pipe, 1.1 and 1.3 for the
// result before, 0.9 and 0.6 for memory, 0.7 and 0.9 at the barriers.  Weights need one
// maximum per tile, and a block for each: 64 x 2048 x 2048 in 119 us, 6.8 TB/s.
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
  int32_t M, K, E, k_tiles, col_blocks, tiles;
};

template <bool KEPT>
struct QuantShared {
  // two tiles of values, or of codes and their rows' scales
  uint8_t in[2][kBlock8][kBlock8 * (KEPT ? 1 : 2)];
  float in_s[2][KEPT ? kBlock8 : 4];
  float part[kQuantWarps][kBlock8];  // maxima that each warp found of its rows
  float r[kBlock8], lo[KEPT ? 4 : kBlock8];  // what the columns' codes are made with
};

// Half-precision pairs as fp32: exact.
__device__ __forceinline__ float2 floats_of(uint32_t h) {
  float2 f;
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(f.x), "=f"(f.y) : "r"(h));
  return f;
}

// One tile, from shared memory.  A warp has rows 16 w .. 16 w + 15 of it: its
// lower half-warp the first eight, the upper one the others, a lane eight columns
// of each.  WHOLE: the tile's 128 columns are all there.
template <bool KEPT, bool ROWS, bool COLS, bool WHOLE>
__device__ __forceinline__ void quant_tile(const QuantP& p, QuantShared<KEPT>& sh, int buf, const RowTile& t, int32_t tile, int32_t kt) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c8 = lane & 15;
  const int row0 = warp * 16 + (lane >> 4) * kRowsPerLane;
  const int32_t k = kt * kBlock8 + c8 * 8, left = WHOLE ? 8 : p.K - k;  // of the row from this lane's columns on
  const int32_t rows = t.r1 - t.r0 - row0;
  uint4 w[kRowsPerLane];  // bf16, or the codes' values as half precision, exact
  float s[kRowsPerLane];  // and their scales
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i) {
    if (KEPT) {
      const uint2 c = *reinterpret_cast<const uint2*>(&sh.in[buf][row0 + i][c8 * 8]);
      asm("{.reg .b16 a, b, c, d; mov.b32 {a, b}, %4; mov.b32 {c, d}, %5;\n"
          " cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; cvt.rn.f16x2.e4m3x2 %2, c; cvt.rn.f16x2.e4m3x2 %3, d;}"
          : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
          : "r"(c.x), "r"(c.y));
      s[i] = sh.in_s[buf][KEPT ? row0 + i : 0];
    } else {
      w[i] = *reinterpret_cast<const uint4*>(&sh.in[buf][row0 + i][c8 * 16]);
    }
  }
  auto value = [&](int i) {
    if (!KEPT) return pairs(w[i]);
    const uint32_t h[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    F8 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v.v[j] = mul_2(floats_of(h[j]), both(s[i]));
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
    const Fit8 f = fit8<true>(mine);
    if (c8 < kRowsPerLane && c8 < rows) p.s[int64_t(kt) * p.M + t.r0 + row0 + c8] = f.s;
    uint8_t* out = p.q + int64_t(t.r0 + row0) * p.ld_q + k;
#pragma unroll
    for (int i = 0; i < kRowsPerLane; ++i) {
      const float r = __shfl_sync(0xFFFFFFFFu, f.r, i, 16), lo = __shfl_sync(0xFFFFFFFFu, f.lo, i, 16);
      if (i < rows && left > 0) put_bytes8(out, left, codes8(pairs(w[i]), r, lo));
      out += p.ld_q;
    }
  }
  if (!COLS || tile >= p.col_blocks) return;  // the same for the whole block
  if (!t.cols) {                              // rows of no expert: their blocks are zeros
#pragma unroll
    for (int i = 0; i < kRowsPerLane; ++i) w[i] = make_uint4(0, 0, 0, 0), s[i] = 0.0f;
  }
  float m[8];
  if (KEPT) {
#pragma unroll
    for (int i = 0; i < kRowsPerLane; ++i) {
      const F8 v = value(i);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = fabsf(j & 1 ? v.v[j / 2].y : v.v[j / 2].x);
        m[j] = i == 0 ? a : max_nan(m[j], a);
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
    float4* o = reinterpret_cast<float4*>(&sh.part[warp][c8 * 8]);
    o[0] = make_float4(m[0], m[1], m[2], m[3]);
    o[1] = make_float4(m[4], m[5], m[6], m[7]);
  }
  __syncthreads();
  if (threadIdx.x < kBlock8) {
    float a = sh.part[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < kQuantWarps; ++i) a = max_nan(a, sh.part[i][threadIdx.x]);
    const Fit8 f = fit8<!KEPT>(a);
    sh.r[threadIdx.x] = f.r;
    if (!KEPT) sh.lo[threadIdx.x] = f.lo;
    if (WHOLE || kt * kBlock8 + int32_t(threadIdx.x) < p.K) p.sc[int64_t(tile) * p.K + kt * kBlock8 + threadIdx.x] = f.s;
  }
  __syncthreads();
  uint8_t* out = p.qc + (int64_t(tile) * kBlock8 + row0) * p.ld_qc + k;
  float2 r[4], lo[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r[j] = *reinterpret_cast<const float2*>(&sh.r[c8 * 8 + 2 * j]);
    if (!KEPT) lo[j] = *reinterpret_cast<const float2*>(&sh.lo[c8 * 8 + 2 * j]);
  }
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i) {
    if (left > 0) put_bytes8(out, left, KEPT ? codes8(value(i), r) : codes8(value(i), r, lo));
    out += p.ld_qc;
  }
}

template <bool KEPT, bool ROWS, bool COLS>
__global__ void __launch_bounds__(kQuantWarps * 32, 3) quant8_kernel(const __grid_constant__ QuantP p) {
  extern __shared__ __align__(16) uint8_t raw[];
  QuantShared<KEPT>& sh = *reinterpret_cast<QuantShared<KEPT>*>(raw);
  constexpr int kThreads = kQuantWarps * 32, kSize = KEPT ? 1 : 2, kPieces = kBlock8 * kSize / 16;  // of a row, 16 bytes each
  constexpr int kStep8 = kThreads / kPieces;  // rows that the block copies at once
  const int copy_row = threadIdx.x / kPieces, copy_at = (threadIdx.x % kPieces) * 16;
  const uint8_t* src = KEPT ? p.xq : reinterpret_cast<const uint8_t*>(p.x);
  const int64_t ld = KEPT ? p.ld_xq : 2 * p.ld_x;
  after_previous();
  // rows that no tile has, and columns past K, are zeros
  auto load = [&](const RowTile& t, int32_t kt, int buf) {
    const int32_t rows = ROWS || t.cols ? t.r1 - t.r0 : 0;
    const uint32_t n = uint32_t(max(0, min(16, (p.K - kt * kBlock8) * kSize - copy_at)));  // bytes
    const uint8_t* from = src + int64_t(t.r0 + copy_row) * ld + int64_t(kt) * kBlock8 * kSize + copy_at;
#pragma unroll
    for (int j = 0; j < kBlock8 / kStep8; ++j) {
      const bool there = copy_row + j * kStep8 < rows && n > 0;
      copy16(&sh.in[buf][copy_row + j * kStep8][copy_at], there ? from : src, there ? n : 0u);
      from += kStep8 * ld;
    }
    if (KEPT && threadIdx.x < kBlock8) {
      const bool there = int32_t(threadIdx.x) < rows;
      copy4(&sh.in_s[buf][KEPT ? threadIdx.x : 0], p.xs + (there ? int64_t(kt) * p.M + t.r0 + threadIdx.x : 0), there);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int32_t tile = blockIdx.x / p.k_tiles, kt = blockIdx.x - tile * p.k_tiles;
  RowTile t = row_tile(p.offsets, p.E, p.M, tile);
  load(t, kt, 0);
  int buf = 0;
  for (int32_t work = blockIdx.x; work < p.tiles; work += gridDim.x, buf ^= 1) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // this tile is there, and the last one has been read
    const int32_t ahead = work + int32_t(gridDim.x);
    int32_t next_tile = 0, next_kt = 0;
    RowTile next = {0, 0, false};
    if (ahead < p.tiles) {
      next_tile = ahead / p.k_tiles;
      next_kt = ahead - next_tile * p.k_tiles;
      next = next_tile == tile ? t : row_tile(p.offsets, p.E, p.M, next_tile);
      load(next, next_kt, buf ^ 1);
    }
    if ((kt + 1) * kBlock8 <= p.K) quant_tile<KEPT, ROWS, COLS, true>(p, sh, buf, t, tile, kt);
    else quant_tile<KEPT, ROWS, COLS, false>(p, sh, buf, t, tile, kt);
    tile = next_tile, kt = next_kt, t = next;
  }
}

template <bool KEPT, bool ROWS, bool COLS>
cudaError_t launch_quant(const QuantP& p, cudaStream_t s, const DevInfo& d) {
  auto kern = quant8_kernel<KEPT, ROWS, COLS>;
  constexpr int smem = int(sizeof(QuantShared<KEPT>)), kPerSm = 3;  // blocks at once, by registers and shared memory
  static SmemLimit limit;
  const cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, unsigned(p.tiles < kPerSm * d.sms ? p.tiles : kPerSm * d.sms), kQuantWarps * 32, smem, s, p, true);
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
  const Fit8 f = fit8<true>(a);
  if (threadIdx.x == 0) p.s[int64_t(rt) * p.k_tiles + kt] = f.s;
  uint8_t* dst = p.q + e * p.stride_q + int64_t(row0) * p.ld_q + k;
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i)
    if (i < rows && left > 0) put_bytes8(dst + i * p.ld_q, left, codes8(pairs(w[i]), f.r, f.lo));
}

}  // namespace

cudaError_t launch_quant8(const glu_block8_quant_args& a, cudaStream_t s, const DevInfo& d) {
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
  p.tiles = (p.col_blocks + (a.E > 0 && a.q ? 1 : 0)) * p.k_tiles;
  if (a.x == nullptr) return launch_quant<true, false, true>(p, s, d);
  if (a.qc == nullptr) return launch_quant<false, true, false>(p, s, d);
  return a.q == nullptr ? launch_quant<false, false, true>(p, s, d) : launch_quant<false, true, true>(p, s, d);
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
