// The gated activation that keeps gate and up in 8 bits, and its backward from
// those (glu_block8.h).  Bound by HBM: every operand is read and every result
// written once; 16 lanes share a row of 128 columns, eight each.
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

// Forward: a warp takes 2 x kFwdRows rows of a 128-column strip.
constexpr int kFwdRows = 4;

template <int ACT, bool H8>
__global__ void __launch_bounds__(kGluWarps * 32) glu8_kernel(const __grid_constant__ GluP p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c8 = lane & 15;
  const int32_t tile = blockIdx.x / p.k_tiles, kt = blockIdx.x - tile * p.k_tiles;
  const int32_t k = kt * kBlock8 + c8 * 8, left = p.H - k;
  const int64_t row0 = (int64_t(tile) * kGluWarps + warp) * 2 * kFwdRows + (lane >> 4) * kFwdRows;
  const int32_t rows = left > 0 ? int32_t(min(int64_t(p.M) - row0, int64_t(kFwdRows))) : 0;
  uint4 g[kFwdRows], u[kFwdRows];
#pragma unroll
  for (int i = 0; i < kFwdRows; ++i) {
    g[i] = u[i] = make_uint4(0, 0, 0, 0);
    if (i < rows) {
      g[i] = raw8(p.gate + (row0 + i) * p.ld_gate + k, left);
      u[i] = raw8(p.up + (row0 + i) * p.ld_up + k, left);
    }
  }
#pragma unroll
  for (int i = 0; i < kFwdRows; ++i) {
    const F8 gv = pairs(g[i]), uv = pairs(u[i]);
    F8 h;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a0, a1, d;
      act8<ACT>(gv.v[j].x, a0, d);
      act8<ACT>(gv.v[j].y, a1, d);
      h.v[j] = mul_2(make_float2(a0, a1), uv.v[j]);
    }
    const uint32_t a = amax_bits(g[i]), b = amax_bits(u[i]);
    const uint32_t m = row_max2(__vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632)));
    const Fit8 fg = fit8(__uint_as_float(m << 16)), fu = fit8(__uint_as_float(m & 0xFFFF0000u));
    Fit8 fh;
    if (H8) fh = fit8(row_max(amax8(h)));
    if (i >= rows) continue;
    const int64_t r = row0 + i, at = int64_t(kt) * p.M + r;
    put_bytes8(p.gq + r * p.ld_gq + k, left, codes8<true>(gv, fg.r, fg.bad));
    put_bytes8(p.uq + r * p.ld_uq + k, left, codes8<true>(uv, fu.r, fu.bad));
    if (H8) put_bytes8(p.hq + r * p.ld_hq + k, left, codes8<false>(h, fh.r, fh.bad));
    else put8(p.h + r * p.ld_h + k, left, packed(h));
    if (c8 == 0) {
      p.gs[at] = fg.s;
      p.us[at] = fu.s;
      if (H8) p.hs[at] = fh.s;
    }
  }
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
  int32_t M, H, E, k_tiles, col_blocks;
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
    act8<ACT>(z.x, a.x, d.x);
    act8<ACT>(z.y, a.y, d.y);
    o.h.v[j] = mul_2(a, w);
    o.du.v[j] = mul_2(dy.v[j], a);
    o.dg.v[j] = mul_2(mul_2(dy.v[j], w), d);
  }
  return o;
}

constexpr int kBwdRows = 4;

template <int ACT>
__global__ void __launch_bounds__(kGluWarps * 32) glu8_bwd_kernel(const __grid_constant__ GluBwdP p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c8 = lane & 15;
  const int32_t tile = blockIdx.x / p.k_tiles, kt = blockIdx.x - tile * p.k_tiles;
  const int32_t k = kt * kBlock8 + c8 * 8, left = p.H - k;
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
#pragma unroll
  for (int i = 0; i < kBwdRows; ++i) {
    if (i >= rows) break;
    const Grads o = glu_grads<ACT>(g[i], gs[i], u[i], us[i], dh[i]);
    const int64_t r = row0 + i;
    uint16_t* d = p.d + r * p.ld_d + k;
    put8(d, left, packed(o.dg));
    // dUp begins at column H, on 16 bytes only where H is a multiple of eight
    if (p.H % 8 == 0) {
      put8(d + p.H, left, packed(o.du));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) d[p.H + j] = bits_of_bf16(j & 1 ? o.du.v[j / 2].y : o.du.v[j / 2].x);
    }
    if (p.h) put8(p.h + r * p.ld_h + k, left, packed(o.h));
  }
}

// Backward, quantised: a block of 16 warps takes 128 rows by 128 columns, a lane
// four rows of eight columns, and holds the three results of its 32 elements in
// registers while the maxima of their columns are found.
constexpr int kTileWarps = 16, kTileRows = 4;

struct TileFits {
  float part[3][kTileWarps][kBlock8];
  float r[3][kBlock8];
  uint32_t bad[3][kBlock8 / 4];
};

template <int ACT>
__global__ void __launch_bounds__(kTileWarps * 32, 1) glu8_bwd_tile_kernel(const __grid_constant__ GluBwdP p) {
  __shared__ TileFits fits;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c8 = lane & 15;
  const int32_t tile = blockIdx.x / p.k_tiles, kt = blockIdx.x - tile * p.k_tiles;
  const RowTile t = row_tile(p.offsets, p.E, p.M, tile);
  const int32_t k = kt * kBlock8 + c8 * 8;
  const int32_t row0 = warp * 8 + (lane >> 4) * kTileRows, rows = t.r1 - t.r0 - row0;
  uint2 g[kTileRows], u[kTileRows];
  uint4 dh[kTileRows];
  float gs[kTileRows], us[kTileRows];
#pragma unroll
  for (int i = 0; i < kTileRows; ++i) {
    g[i] = u[i] = make_uint2(0, 0);
    dh[i] = make_uint4(0, 0, 0, 0);
    gs[i] = us[i] = 0.0f;
    if (i < rows) {
      const int64_t r = t.r0 + row0 + i, at = int64_t(kt) * p.M + r;
      g[i] = bytes8(p.gq + r * p.ld_gq + k, 8);
      u[i] = bytes8(p.uq + r * p.ld_uq + k, 8);
      dh[i] = ldg_once(p.dh + r * p.ld_dh + k);
      gs[i] = __ldg(p.gs + at);
      us[i] = __ldg(p.us + at);
    }
  }
  F8 v[3][kTileRows];
#pragma unroll
  for (int i = 0; i < kTileRows; ++i) {
    const Grads o = glu_grads<ACT>(g[i], gs[i], u[i], us[i], dh[i]);
    v[0][i] = o.dg;
    v[1][i] = o.du;
    v[2][i] = o.h;
  }
  // rows of d: lane 2 i + x of a half fits row i of dGate (x = 0) or dUp
  float mine = 0.0f;
#pragma unroll
  for (int i = 0; i < kTileRows; ++i)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float m = row_max(amax8(v[x][i]));
      if (c8 == 2 * i + x) mine = m;
    }
  const Fit8 f = fit8(mine);
  if (c8 < 2 * kTileRows && c8 / 2 < rows)
    p.ds[int64_t(kt + (c8 & 1) * p.k_tiles) * p.M + t.r0 + row0 + c8 / 2] = f.s;
#pragma unroll
  for (int i = 0; i < kTileRows; ++i)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float r = __shfl_sync(0xFFFFFFFFu, f.r, 2 * i + x, 16);
      const uint32_t bad = __shfl_sync(0xFFFFFFFFu, f.bad, 2 * i + x, 16);
      if (i < rows) put_bytes8(p.dq + (t.r0 + row0 + i) * p.ld_dq + x * p.H + k, 8, codes8<false>(v[x][i], r, bad));
    }
  if (tile >= p.col_blocks) return;
  if (!t.cols) {  // rows of no expert: their blocks are zeros
#pragma unroll
    for (int x = 0; x < 3; ++x)
#pragma unroll
      for (int i = 0; i < kTileRows; ++i) v[x][i] = zeros();
  }
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    float m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = 0.0f;
#pragma unroll
      for (int i = 0; i < kTileRows; ++i) m[j] = max_nan(m[j], fabsf(j & 1 ? v[x][i].v[j / 2].y : v[x][i].v[j / 2].x));
      m[j] = max_nan(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], 16));
    }
    if (lane < 16) {
      float4* o = reinterpret_cast<float4*>(&fits.part[x][warp][c8 * 8]);
      o[0] = make_float4(m[0], m[1], m[2], m[3]);
      o[1] = make_float4(m[4], m[5], m[6], m[7]);
    }
  }
  __syncthreads();
  if (threadIdx.x < 3 * kBlock8) {
    const int x = threadIdx.x / kBlock8, c = threadIdx.x % kBlock8;
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < kTileWarps; ++i) a = max_nan(a, fits.part[x][i][c]);
    const Fit8 fc = fit8(a);
    fits.r[x][c] = fc.r;
    reinterpret_cast<uint8_t*>(fits.bad[x])[c] = uint8_t(fc.bad);
    if (x < 2) p.dsc[int64_t(tile) * 2 * p.H + x * p.H + kt * kBlock8 + c] = fc.s;
    else if (p.hsc) p.hsc[int64_t(tile) * p.H + kt * kBlock8 + c] = fc.s;
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    if (x == 2 && p.hqc == nullptr) break;
    float2 r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = *reinterpret_cast<const float2*>(&fits.r[x][c8 * 8 + 2 * j]);
    const uint2 bad = *reinterpret_cast<const uint2*>(&fits.bad[x][c8 * 2]);
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
      uint2 o = codes8<false>(v[x][i], r);
      o.x |= bad.x, o.y |= bad.y;
      const int64_t row = int64_t(tile) * kBlock8 + row0 + i;
      put_bytes8(x < 2 ? p.dqc + row * p.ld_dqc + x * p.H + k : p.hqc + row * p.ld_hqc + k, 8, o);
    }
  }
}

template <int ACT>
cudaError_t launch_fwd(const GluP& p, cudaStream_t s) {
  const int64_t per = kGluWarps * 2 * kFwdRows, tiles = (p.M + per - 1) / per * p.k_tiles;
  if (p.hq) glu8_kernel<ACT, true><<<unsigned(tiles), kGluWarps * 32, 0, s>>>(p);
  else glu8_kernel<ACT, false><<<unsigned(tiles), kGluWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}
template <int ACT>
cudaError_t launch_bwd(const GluBwdP& p, cudaStream_t s) {
  if (p.d) {
    const int64_t per = kGluWarps * 2 * kBwdRows, tiles = (p.M + per - 1) / per * p.k_tiles;
    glu8_bwd_kernel<ACT><<<unsigned(tiles), kGluWarps * 32, 0, s>>>(p);
  } else {
    const int64_t tiles = int64_t(p.col_blocks + (p.E > 0 ? 1 : 0)) * p.k_tiles;
    glu8_bwd_tile_kernel<ACT><<<unsigned(tiles), kTileWarps * 32, 0, s>>>(p);
  }
  return cudaGetLastError();
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

cudaError_t launch_glu8_bwd(const glu_block8_glu_bwd_args& a, cudaStream_t s) {
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
    case GLU_ACT_SILU: return launch_bwd<GLU_ACT_SILU>(p, s);
    case GLU_ACT_GELU_TANH: return launch_bwd<GLU_ACT_GELU_TANH>(p, s);
    case GLU_ACT_RELU: return launch_bwd<GLU_ACT_RELU>(p, s);
    case GLU_ACT_GELU_ERF: return launch_bwd<GLU_ACT_GELU_ERF>(p, s);
    default: return launch_bwd<GLU_ACT_IDENTITY>(p, s);
  }
}

}  // namespace gq
