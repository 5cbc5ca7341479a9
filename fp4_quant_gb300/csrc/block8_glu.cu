// The gated activation that keeps gate and up in 8 bits, and its backward from
// those (glu_block8.h).  Every operand is read and every result written once; 16
// lanes share a row of 128 columns, eight each.  Forward takes about 30 instructions
// per value (calls of 39.2 us for 4096 x 7168, 5.3 TB/s), the quantised backward 40
// per place of a tile (80.2 us for 32768 x 1024 of 64 experts).  The bf16 one takes
// 27.5 us for 8191 x 1462, where dUp's rows begin inside 16 bytes, and three quarters of
// that for a width of 1464.  No unit is full: in that order warps issue in 64, 58 and
// 62 % of the cycles, the integer pipe works in 49, 51 and 41 %, DRAM in 53, 26 and
// 29 %.  Of the 10.6, 6.9 and 8.2 cycles between a warp's instructions it waits for loads
// most where the kernel has no copies ahead (4.1 forward, 2.3 in the bf16 backward); the
// quantised backward, four warps per scheduler, waits 1.2 for the result before, 0.9
// each for the pipe and for shared memory and 0.7 at the barriers.
#include "block8_act.cuh"

namespace gq {
namespace {

constexpr int kGluWarps = 8;

struct GluP {
  const uint16_t *gate, *up;
  uint16_t* h;
  uint8_t *hq, *gq, *uq;
  float *hs, *gs, *us;
  int64_t ld_gate, ld_up, ld_h, ld_hq, ld_gq, ld_uq;
  int32_t M, H, k_tiles;
};

// Forward: a warp takes 2 x kFwdRows rows of a 128-column strip (four rows per
// lane: 53 us, two, with four blocks per SM: 45, in isolation).
constexpr int kFwdRows = 2;

// WHOLE (here and below): the strip's 128 columns are all there.
template <int ACT, bool H8, bool WHOLE>
__device__ __forceinline__ void glu_tile(const GluP& p, int32_t tile, int32_t kt) {
  constexpr bool kExact = ACT == GLU_ACT_RELU || ACT == GLU_ACT_IDENTITY;  // h is a product of two bf16, not rounded
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c8 = lane & 15;
  const int32_t k = kt * kBlock8 + c8 * 8, left = WHOLE ? 8 : p.H - k;
  const int64_t row0 = (int64_t(tile) * kGluWarps + warp) * 2 * kFwdRows + (lane >> 4) * kFwdRows;
  const int32_t have = int32_t(min(int64_t(p.M) - row0, int64_t(kFwdRows))), rows = left > 0 ? have : 0;
  uint4 g[kFwdRows], u[kFwdRows];
#pragma unroll
  for (int i = 0; i < kFwdRows; ++i) {
    g[i] = u[i] = make_uint4(0, 0, 0, 0);
    if (i < rows) {
      g[i] = raw8(p.gate + (row0 + i) * p.ld_gate + k, left);
      u[i] = raw8(p.up + (row0 + i) * p.ld_up + k, left);
    }
  }
  // the blocks' maxima: of gate, up and h of row i as values 4 i, 4 i + 1, 4 i + 2,
  // which lanes of that number fit
  F8 h[kFwdRows];
  float m[4 * kFwdRows];
#pragma unroll
  for (int i = 0; i < kFwdRows; ++i) {
    const F8 gv = pairs(g[i]), uv = pairs(u[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float2 a, d;
      act8<ACT>(gv.v[j], a, d);
      h[i].v[j] = mul_2(a, uv.v[j]);
    }
    m[4 * i] = top_half(amax_bits(g[i]));
    m[4 * i + 1] = top_half(amax_bits(u[i]));
    m[4 * i + 2] = H8 ? amax8(h[i]) : 0.0f;
    m[4 * i + 3] = 0.0f;
  }
  const Fit8 f = fit8<true>(scatter_max(m, lane));
  {
    float* s = (c8 & 3) == 0 ? p.gs : (c8 & 3) == 1 ? p.us : H8 && (c8 & 3) == 2 ? p.hs : nullptr;
    if (s && c8 < 4 * kFwdRows && c8 / 4 < have) s[int64_t(kt) * p.M + row0 + c8 / 4] = f.s;
  }
#pragma unroll
  for (int i = 0; i < kFwdRows; ++i) {
    const float rg = __shfl_sync(0xFFFFFFFFu, f.r, 4 * i, 16), lg = __shfl_sync(0xFFFFFFFFu, f.lo, 4 * i, 16);
    const float ru = __shfl_sync(0xFFFFFFFFu, f.r, 4 * i + 1, 16), lu = __shfl_sync(0xFFFFFFFFu, f.lo, 4 * i + 1, 16);
    const float rh = H8 ? __shfl_sync(0xFFFFFFFFu, kExact ? f.r : f.r + f.lo, 4 * i + 2, 16) : 0.0f;
    const float lh = H8 && kExact ? __shfl_sync(0xFFFFFFFFu, f.lo, 4 * i + 2, 16) : 0.0f;
    if (i >= rows) continue;
    const int64_t r = row0 + i;
    put_bytes8(p.gq + r * p.ld_gq + k, left, codes8(pairs(g[i]), rg, lg));
    put_bytes8(p.uq + r * p.ld_uq + k, left, codes8(pairs(u[i]), ru, lu));
    if (H8) put_bytes8(p.hq + r * p.ld_hq + k, left, kExact ? codes8(h[i], rh, lh) : codes8(h[i], rh));
    else put8(p.h + r * p.ld_h + k, left, packed(h[i]));
  }
}

template <int ACT, bool H8>
__global__ void __launch_bounds__(kGluWarps * 32, 4) glu8_kernel(const __grid_constant__ GluP p) {
  const int32_t tile = blockIdx.x / p.k_tiles, kt = blockIdx.x - tile * p.k_tiles;
  after_previous();
  if ((kt + 1) * kBlock8 <= p.H) glu_tile<ACT, H8, true>(p, tile, kt);
  else glu_tile<ACT, H8, false>(p, tile, kt);
}

struct GluBwdP {
  const uint8_t *gq, *uq;
  const float *gs, *us;
  const uint16_t* dh;
  const int32_t* offsets;
  uint16_t *d, *h;
  uint8_t *dq, *dqc, *hqc;
  float *ds, *dsc, *hsc;
  int64_t ld_gq, ld_uq, ld_dh, ld_d, ld_h, ld_dq, ld_dqc, ld_hqc;
  int32_t M, H, E, k_tiles, col_blocks, tiles;
};

struct Grads {
  F8 dg, du, h;
};
template <int ACT>
__device__ __forceinline__ Grads glu_grads(const uint2& gq, float gs, const uint2& uq, float us, const uint4& dh) {
  Grads o;
  const F8 g = values8(gq), u = values8(uq), dy = pairs(dh);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 z = mul_2(g.v[j], both(gs)), w = mul_2(u.v[j], both(us));
    float2 a, d;
    act8<ACT>(z, a, d);
    o.h.v[j] = mul_2(a, w);
    o.du.v[j] = mul_2(dy.v[j], a);
    o.dg.v[j] = mul_2(mul_2(dy.v[j], w), d);
  }
  return o;
}

// A row's chunks of eight bf16, one per lane of 16 (`left` elements from the lane's
// first on), to where the row begins `off` elements (1 .. 7) behind 16 bytes: a
// lane stores the 16 bytes in which its chunk begins, with the last `off` elements
// of the lane before it, from `buf` (the half-warp's own, four words ahead of the
// row's 64).  What fills no 16 bytes here goes in words or elements.  `row`: the
// lane's first element.  All 32 lanes take part.  WHOLE: the sixteen chunks are
// all there.
template <bool WHOLE>
__device__ __forceinline__ void put_shifted(uint16_t* row, int off, int left, bool store, const uint4& v, int c8, uint32_t* buf) {
  __syncwarp();
  *reinterpret_cast<uint4*>(buf + 4 + 4 * c8) = v;
  __syncwarp();
  if (!store) return;
  const int n = WHOLE ? 8 : min(left, 8);
  const bool whole = c8 > 0 && n >= 8 - off;
  const uint32_t* from = buf + 4 + 4 * c8 - (off + 1) / 2;
  uint32_t w[5];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = from[j];
  if (off & 1) {
    w[4] = from[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], 16);
  }
  if (whole) stg_once(row - off, make_uint4(w[0], w[1], w[2], w[3]));
  if (WHOLE && off % 2 == 0) {
    // what is left of the first and of the last chunk, (8 - off) / 2 and off / 2 words
    // of the same numbers 0 .. 3: lane c8 < 4 stores word c8
    if (c8 < 4) {
      const int at = c8 < (8 - off) / 2 ? c8 : 60 + c8;  // word of the row
      *reinterpret_cast<uint32_t*>(row - 8 * c8 + 2 * at) = buf[4 + at];
    }
    return;
  }
  // the chunk's elements up to its 16 bytes' end where they were not stored, and
  // those behind it where no lane follows
  const int end = 8 - off;
  const int lo = whole ? end : c8 > 0 ? -off : 0, hi = c8 == 15 || left <= 8 ? n : min(n, end);
  const uint16_t* element = reinterpret_cast<const uint16_t*>(buf + 4 + 4 * c8);
  for (int e = lo; e < hi; ++e) row[e] = element[e];
}

constexpr int kBwdRows = 4;

// 64 words of dUp's chunks per half-warp, and four ahead of them.
using ShiftBuf = uint32_t[2 * kGluWarps][4 + 64];

template <int ACT, bool WHOLE>
__device__ __forceinline__ void glu_bwd_tile(const GluBwdP& p, ShiftBuf& buf, int32_t tile, int32_t kt) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c8 = lane & 15;
  const int32_t k = kt * kBlock8 + c8 * 8, left = WHOLE ? 8 : p.H - k;
  const int64_t row0 = (int64_t(tile) * kGluWarps + warp) * 2 * kBwdRows + (lane >> 4) * kBwdRows;
  const int32_t rows = left > 0 ? int32_t(min(int64_t(p.M) - row0, int64_t(kBwdRows))) : 0;
  uint2 g[kBwdRows], u[kBwdRows];
  uint4 dh[kBwdRows];
  float gs[kBwdRows], us[kBwdRows];
#pragma unroll
  for (int i = 0; i < kBwdRows; ++i) {
    if (i < rows) {
      const int64_t r = row0 + i, at = int64_t(kt) * p.M + r;
      g[i] = bytes8(p.gq + r * p.ld_gq + k, left);
      u[i] = bytes8(p.uq + r * p.ld_uq + k, left);
      dh[i] = raw8(p.dh + r * p.ld_dh + k, left);
      gs[i] = __ldg(p.gs + at);
      us[i] = __ldg(p.us + at);
    }
  }
  const int off = p.H % 8;
#pragma unroll
  for (int i = 0; i < kBwdRows; ++i) {
    const int64_t r = row0 + i;
    const bool store = i < rows;
    uint4 du = make_uint4(0, 0, 0, 0);
    if (store) {
      const Grads o = glu_grads<ACT>(g[i], gs[i], u[i], us[i], dh[i]);
      put8(p.d + r * p.ld_d + k, left, packed(o.dg));
      du = packed(o.du);
      if (off == 0) put8(p.d + r * p.ld_d + p.H + k, left, du);
      if (p.h) put8(p.h + r * p.ld_h + k, left, packed(o.h));
    }
    if (off != 0) put_shifted<WHOLE>(p.d + r * p.ld_d + p.H + k, off, WHOLE ? p.H - k : left, store, du, c8, buf[2 * warp + (lane >> 4)]);
  }
}

template <int ACT>
__global__ void __launch_bounds__(kGluWarps * 32, 3) glu8_bwd_kernel(const __grid_constant__ GluBwdP p) {
  __shared__ __align__(16) ShiftBuf buf;
  const int32_t tile = blockIdx.x / p.k_tiles, kt = blockIdx.x - tile * p.k_tiles;
  after_previous();
  if ((kt + 1) * kBlock8 <= p.H) glu_bwd_tile<ACT, true>(p, buf, tile, kt);
  else glu_bwd_tile<ACT, false>(p, buf, tile, kt);
}

// Backward, quantised: blocks of 16 warps, one per SM, walk tiles of 128 rows by
// 128 columns.  A lane has four rows of eight columns, and holds the three results
// of its 32 elements in registers while the maxima of rows and columns are found;
// the next tile's operands are on their way into shared memory meanwhile (a block
// per tile: 113 us for 32768 x 1024, this way 94, with cheaper activations and
// scales 81).
constexpr int kTileWarps = 16, kTileRows = 4;

struct TileIn {
  uint16_t dh[kBlock8][kBlock8];
  uint8_t g[kBlock8][kBlock8], u[kBlock8][kBlock8];
  float gs[kBlock8], us[kBlock8];
};
struct TileShared {
  TileIn in[2];
  float part[3][kTileWarps][kBlock8];
  float r[3][kBlock8];
  int32_t offsets[kMaxExperts + 1];
};

template <int ACT>
__global__ void __launch_bounds__(kTileWarps * 32, 1) glu8_bwd_tile_kernel(const __grid_constant__ GluBwdP p) {
  extern __shared__ __align__(16) uint8_t raw[];
  TileShared& sh = *reinterpret_cast<TileShared*>(raw);
  constexpr int kThreads = kTileWarps * 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c8 = lane & 15;
  const int row0 = warp * 8 + (lane >> 4) * kTileRows;
  after_previous();
  if (p.offsets) {
    for (int e = threadIdx.x; e <= p.E; e += kThreads) sh.offsets[e] = __ldg(p.offsets + e);
    __syncthreads();
  }
  auto rows_of = [&](int32_t w) { return row_tile(p.offsets ? sh.offsets : nullptr, p.E, p.M, w / p.k_tiles); };
  auto load = [&](int32_t w, const RowTile& t, TileIn& in) {
    const int32_t kt = w % p.k_tiles, k = kt * kBlock8, rows = t.r1 - t.r0;
    // a warp copies the eight rows that it will read; rows of no tile are not read
    // (their first row's address stands in)
    const int first = warp * 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = first + 2 * j + (lane >> 4), c = (lane & 15) * 8;
      copy16(&in.dh[r][c], p.dh + int64_t(r < rows ? t.r0 + r : 0) * p.ld_dh + k + c, r < rows ? 16u : 0u);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = first + 4 * j + (lane >> 3), c = (lane & 7) * 16;
      const int64_t m = r < rows ? t.r0 + r : 0;
      copy16(&in.g[r][c], p.gq + m * p.ld_gq + k + c, r < rows ? 16u : 0u);
      copy16(&in.u[r][c], p.uq + m * p.ld_uq + k + c, r < rows ? 16u : 0u);
    }
    if (lane < 16) {
      const int r = first + (lane & 7);
      const float* s = (lane < 8 ? p.gs : p.us) + int64_t(kt) * p.M + (r < rows ? t.r0 + r : 0);
      copy4(lane < 8 ? &in.gs[r] : &in.us[r], s, r < rows);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  RowTile t = {0, 0, false};
  if (int32_t(blockIdx.x) < p.tiles) {
    t = rows_of(blockIdx.x);
    load(blockIdx.x, t, sh.in[0]);
  }
  int buf = 0;
  for (int32_t w = blockIdx.x; w < p.tiles; w += gridDim.x, buf ^= 1) {
    RowTile next = {0, 0, false};
    if (w + int32_t(gridDim.x) < p.tiles) {
      next = rows_of(w + gridDim.x);
      load(w + gridDim.x, next, sh.in[buf ^ 1]);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncwarp();  // the other lanes' copies
    const TileIn& in = sh.in[buf];
    const int32_t tile = w / p.k_tiles, kt = w - tile * p.k_tiles, k = kt * kBlock8 + c8 * 8, rows = t.r1 - t.r0 - row0;
    F8 v[3][kTileRows];
    if (t.r1 - t.r0 > warp * 8) {
      float m[2 * kTileRows];
#pragma unroll
      for (int i = 0; i < kTileRows; ++i) {
        const int r = row0 + i;
        const Grads o = glu_grads<ACT>(*reinterpret_cast<const uint2*>(&in.g[r][c8 * 8]), in.gs[r], *reinterpret_cast<const uint2*>(&in.u[r][c8 * 8]),
                                       in.us[r], *reinterpret_cast<const uint4*>(&in.dh[r][c8 * 8]));
        v[0][i] = o.dg;
        v[1][i] = o.du;
        v[2][i] = o.h;
        m[2 * i] = amax8(o.dg);
        m[2 * i + 1] = amax8(o.du);
      }
      // rows of d: lane 2 i + x of eight fits row i of dGate (x = 0) or dUp
      const Fit8 f = fit8<false>(scatter_max(m, lane));
      if (c8 < 2 * kTileRows && c8 / 2 < rows) p.ds[int64_t(kt + (c8 & 1) * p.k_tiles) * p.M + t.r0 + row0 + c8 / 2] = f.s;
#pragma unroll
      for (int i = 0; i < kTileRows; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float r = __shfl_sync(0xFFFFFFFFu, f.r, 2 * i + x, 16);
          if (i < rows) put_bytes8(p.dq + (t.r0 + row0 + i) * p.ld_dq + x * p.H + k, 8, codes8(v[x][i], r));
        }
    } else {  // none of the warp's rows: zeros, for the columns
#pragma unroll
      for (int x = 0; x < 3; ++x)
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) v[x][i] = zeros();
    }
    if (tile < p.col_blocks) {  // the same for the whole block
      if (!t.cols) {  // rows of no expert: their blocks are zeros
#pragma unroll
        for (int x = 0; x < 3; ++x)
#pragma unroll
          for (int i = 0; i < kTileRows; ++i) v[x][i] = zeros();
      }
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        float c[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          auto at = [&](int i) { return fabsf(j & 1 ? v[x][i].v[j / 2].y : v[x][i].v[j / 2].x); };
          c[j] = max_nan(max_nan(at(0), at(1)), max_nan(at(2), at(3)));
        }
        // the half-warps' maxima: a lane of each keeps four columns
        const bool up = lane & 16;
        float o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float got = __shfl_xor_sync(0xFFFFFFFFu, up ? c[j] : c[4 + j], 16);
          o[j] = max_nan(up ? c[4 + j] : c[j], got);
        }
        *reinterpret_cast<float4*>(&sh.part[x][warp][c8 * 8 + (up ? 4 : 0)]) = make_float4(o[0], o[1], o[2], o[3]);
      }
      __syncthreads();
      if (threadIdx.x < 3 * kBlock8) {
        const int x = threadIdx.x / kBlock8, c = threadIdx.x % kBlock8;
        float a = sh.part[x][0][c];
#pragma unroll
        for (int i = 1; i < kTileWarps; ++i) a = max_nan(a, sh.part[x][i][c]);
        const Fit8 fc = fit8<false>(a);
        sh.r[x][c] = fc.r;
        if (x < 2) p.dsc[int64_t(tile) * 2 * p.H + x * p.H + kt * kBlock8 + c] = fc.s;
        else if (p.hsc) p.hsc[int64_t(tile) * p.H + kt * kBlock8 + c] = fc.s;
      }
      __syncthreads();
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        if (x == 2 && p.hqc == nullptr) break;
        float2 r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = *reinterpret_cast<const float2*>(&sh.r[x][c8 * 8 + 2 * j]);
        const int64_t row = int64_t(tile) * kBlock8 + row0;
        uint8_t* out = x < 2 ? p.dqc + row * p.ld_dqc + x * p.H + k : p.hqc + row * p.ld_hqc + k;
        const int64_t ld = x < 2 ? p.ld_dqc : p.ld_hqc;
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) put_bytes8(out + i * ld, 8, codes8(v[x][i], r));
      }
    }
    __syncwarp();  // the warp has read its rows before those of the next tile but one arrive
    t = next;
  }
}

template <int ACT>
cudaError_t launch_fwd(const GluP& p, cudaStream_t s) {
  const int64_t per = kGluWarps * 2 * kFwdRows, tiles = (p.M + per - 1) / per * p.k_tiles;
  return launch_kernel(p.hq ? glu8_kernel<ACT, true> : glu8_kernel<ACT, false>, unsigned(tiles), kGluWarps * 32, 0, s, p, true);
}
template <int ACT>
cudaError_t launch_bwd(GluBwdP& p, cudaStream_t s, const DevInfo& d) {
  if (p.d) {
    const int64_t per = kGluWarps * 2 * kBwdRows, tiles = (p.M + per - 1) / per * p.k_tiles;
    return launch_kernel(glu8_bwd_kernel<ACT>, unsigned(tiles), kGluWarps * 32, 0, s, p, true);
  } else {
    p.tiles = (p.col_blocks + (p.E > 0 ? 1 : 0)) * p.k_tiles;
    auto kern = glu8_bwd_tile_kernel<ACT>;
    static SmemLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern), int(sizeof(TileShared)));
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, unsigned(p.tiles < d.sms ? p.tiles : d.sms), kTileWarps * 32, sizeof(TileShared), s, p, true);
  }
}

}  // namespace

cudaError_t launch_glu8(const glu_block8_glu_args& a, cudaStream_t s) {
  GluP p;
  p.gate = static_cast<const uint16_t*>(a.gate);
  p.up = static_cast<const uint16_t*>(a.up);
  p.h = static_cast<uint16_t*>(a.h);
  p.hq = static_cast<uint8_t*>(a.hq);
  p.gq = static_cast<uint8_t*>(a.gq);
  p.uq = static_cast<uint8_t*>(a.uq);
  p.hs = a.hs;
  p.gs = a.gs;
  p.us = a.us;
  p.ld_gate = a.ld_gate;
  p.ld_up = a.ld_up;
  p.ld_h = a.ld_h;
  p.ld_hq = a.ld_hq;
  p.ld_gq = a.ld_gq;
  p.ld_uq = a.ld_uq;
  p.M = int32_t(a.M);
  p.H = int32_t(a.H);
  p.k_tiles = int32_t(blocks8(a.H));
  switch (a.act) {
    case GLU_ACT_SILU: return launch_fwd<GLU_ACT_SILU>(p, s);
    case GLU_ACT_GELU_TANH: return launch_fwd<GLU_ACT_GELU_TANH>(p, s);
    case GLU_ACT_RELU: return launch_fwd<GLU_ACT_RELU>(p, s);
    case GLU_ACT_GELU_ERF: return launch_fwd<GLU_ACT_GELU_ERF>(p, s);
    default: return launch_fwd<GLU_ACT_IDENTITY>(p, s);
  }
}

cudaError_t launch_glu8_bwd(const glu_block8_glu_bwd_args& a, cudaStream_t s, const DevInfo& d) {
  GluBwdP p;
  p.gq = static_cast<const uint8_t*>(a.gq);
  p.uq = static_cast<const uint8_t*>(a.uq);
  p.gs = a.gs;
  p.us = a.us;
  p.dh = static_cast<const uint16_t*>(a.dh);
  p.offsets = a.E > 0 ? a.offsets : nullptr;
  p.d = static_cast<uint16_t*>(a.d);
  p.h = static_cast<uint16_t*>(a.h);
  p.dq = static_cast<uint8_t*>(a.dq);
  p.dqc = static_cast<uint8_t*>(a.dqc);
  p.hqc = static_cast<uint8_t*>(a.hqc);
  p.ds = a.ds;
  p.dsc = a.dsc;
  p.hsc = a.hsc;
  p.ld_gq = a.ld_gq;
  p.ld_uq = a.ld_uq;
  p.ld_dh = a.ld_dh;
  p.ld_d = a.ld_d;
  p.ld_h = a.ld_h;
  p.ld_dq = a.ld_dq;
  p.ld_dqc = a.ld_dqc;
  p.ld_hqc = a.ld_hqc;
  p.M = int32_t(a.M);
  p.H = int32_t(a.H);
  p.E = a.E;
  p.k_tiles = int32_t(blocks8(a.H));
  p.col_blocks = int32_t(col_blocks8(a.M, a.E));
  switch (a.act) {
    case GLU_ACT_SILU: return launch_bwd<GLU_ACT_SILU>(p, s, d);
    case GLU_ACT_GELU_TANH: return launch_bwd<GLU_ACT_GELU_TANH>(p, s, d);
    case GLU_ACT_RELU: return launch_bwd<GLU_ACT_RELU>(p, s, d);
    case GLU_ACT_GELU_ERF: return launch_bwd<GLU_ACT_GELU_ERF>(p, s, d);
    default: return launch_bwd<GLU_ACT_IDENTITY>(p, s, d);
  }
}

}  // namespace gq
