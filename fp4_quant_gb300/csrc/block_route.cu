// Tokens sorted by expert and back (glu_block.h): the stable sort of the
// assignments, and the rows moved by it.
//
// The sort counts: with h[b][e] the assignments of expert e in block b of
// the list, assignment j of block b goes to
//   offsets[e] + sum over b' < b of h[b'][e] + (its rank among e's in block b),
// which keeps the order inside an expert and has one answer, whatever the
// order in which the blocks run.  It moves 12 bytes per assignment next to
// the rows' 2 D bytes.
//
// The rows are bound by DRAM: dispatch and combine_bwd write every row of
// the sorted matrix, combine and combine_bwd read every kept one, and each
// token's own row is read or written once, by one warp.  16384 tokens with eight
// rows of 2048 each: dispatch 97 us (6.2 TB/s), combine 89 us, combine_bwd 180
// us (6.2 TB/s); the sort of their 131072 assignments 12 us.
#include "block.h"
#include "block_util.cuh"

namespace gq {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int64_t kSortMin = 1024;  // assignments per block of the list, at least
constexpr int64_t kSortBlocks = 1024;

struct RouteP {
  const void* ids;
  int32_t *slot, *src, *offsets, *hist;  // hist [blocks, E]
  int64_t n, per_block;
  int32_t E, id_bytes, blocks;
};

__device__ __forceinline__ int id_at(const RouteP& p, int64_t j) {
  const int64_t v = p.id_bytes == 8 ? static_cast<const int64_t*>(p.ids)[j] : static_cast<const int32_t*>(p.ids)[j];
  return v >= 0 && v < p.E ? int(v) : -1;
}

__global__ void __launch_bounds__(kSortThreads) route_count_kernel(const RouteP p) {
  __shared__ int32_t h[kMaxExperts];
  after_previous();
  for (int e = threadIdx.x; e < p.E; e += kSortThreads) h[e] = 0;
  __syncthreads();
  const int64_t j0 = int64_t(blockIdx.x) * p.per_block, j1 = min(p.n, j0 + p.per_block);
  for (int64_t j = j0 + threadIdx.x; j < j1; j += kSortThreads) {
    const int e = id_at(p, j);
    if (e >= 0) atomicAdd(&h[e], 1);  // whole numbers: the order does not matter
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kSortThreads) p.hist[int64_t(blockIdx.x) * p.E + e] = h[e];
}

// Inclusive sum over the block of one value per thread (kSortThreads of them).
__device__ __forceinline__ int32_t block_scan(int32_t v, int32_t* warp_total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_total[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int32_t t = warp_total[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t u = __shfl_up_sync(0xFFFFFFFFu, t, o);
      if (lane >= o) t += u;
    }
    warp_total[lane] = t;
  }
  __syncthreads();
  return v + (warp ? warp_total[warp - 1] : 0);
}

// Places of block b's assignments.  `count` (shared, [warps, E]) holds each
// warp's count of each expert, then its start.  A list of one block is counted
// here too.
__global__ void __launch_bounds__(kSortThreads) route_place_kernel(const RouteP p) {
  __shared__ int32_t base[kMaxExperts + 1];  // next place of each expert for this block
  __shared__ int32_t all[kMaxExperts];
  __shared__ int32_t warp_total[32];
  extern __shared__ int32_t count[];  // [kSortWarps][E]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // totals, and what the blocks before this one have of them (whole numbers:
  // the order of the additions does not matter)
  if (int(threadIdx.x) < p.E) all[threadIdx.x] = base[threadIdx.x] = 0;
  after_previous();
  __syncthreads();
  if (p.blocks == 1) {
    for (int64_t j = threadIdx.x; j < p.n; j += kSortThreads) {
      const int e = id_at(p, j);
      if (e >= 0) atomicAdd(&all[e], 1);
    }
  } else {
    const int64_t ahead = int64_t(blockIdx.x) * p.E;
    for (int64_t i = threadIdx.x; i < int64_t(p.blocks) * p.E; i += kSortThreads) {
      const int32_t v = p.hist[i];
      if (v == 0) continue;
      const int e = int(i % p.E);
      atomicAdd(&all[e], v);
      if (i < ahead) atomicAdd(&base[e], v);
    }
  }
  __syncthreads();
  const int32_t total = int(threadIdx.x) < p.E ? all[threadIdx.x] : 0;
  const int32_t end = block_scan(total, warp_total);
  if (int(threadIdx.x) < p.E) {
    base[threadIdx.x] += end - total;
    if (blockIdx.x == 0) p.offsets[threadIdx.x + 1] = end;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) p.offsets[0] = 0;
  if (int(threadIdx.x) == p.E - 1) base[kMaxExperts] = end;  // assignments kept in all
  __syncthreads();
  const int64_t j0 = int64_t(blockIdx.x) * p.per_block, j1 = min(p.n, j0 + p.per_block);
  for (int64_t t0 = j0; t0 < j1; t0 += kSortThreads) {
    for (int i = threadIdx.x; i < kSortWarps * p.E; i += kSortThreads) count[i] = 0;
    __syncthreads();
    const int64_t j = t0 + threadIdx.x;
    const int e = j < j1 ? id_at(p, j) : -2;
    // rank among the lanes of this warp with the same expert
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (e >= 0 && rank == 0) count[warp * p.E + e] = __popc(same);
    __syncthreads();
    // each expert's start in every warp, and its next place after this tile
    for (int x = threadIdx.x; x < p.E; x += kSortThreads) {
      int32_t at = base[x];
      for (int w = 0; w < kSortWarps; ++w) {
        const int32_t v = count[w * p.E + x];
        count[w * p.E + x] = at;
        at += v;
      }
      base[x] = at;
    }
    __syncthreads();
    if (j < j1) {
      const int32_t place = e >= 0 ? count[warp * p.E + e] + rank : -1;
      p.slot[j] = place;
      if (place >= 0) p.src[place] = int32_t(j);
    }
    __syncthreads();
  }
  // the places past the last expert's
  const int64_t kept = base[kMaxExperts];
  for (int64_t i = kept + int64_t(blockIdx.x) * kSortThreads + threadIdx.x; i < p.n; i += int64_t(gridDim.x) * kSortThreads)
    p.src[i] = -1;
}

int64_t sort_per_block(int64_t n) {
  const int64_t per = (n + kSortBlocks - 1) / kSortBlocks;
  return per <= kSortMin ? kSortMin : (per + kSortThreads - 1) / kSortThreads * kSortThreads;
}

// ------------------------------------------------------------------ rows --

struct RowsP {
  int64_t T, K, D, R;
  int64_t ld_tokens, ld_rows, ld_rows_out, ld_residual;
  const int32_t *slot, *src;
  const float* w;
  const uint16_t *tokens_in, *rows_in, *residual;
  uint16_t *tokens_out, *rows_out;
  float* dw;
};

constexpr int kRowWarps = 8;

// Zero rows of the places that no assignment has; warp `wid` of `warps`.
__device__ __forceinline__ void zero_rows(const RowsP& p, int64_t wid, int64_t warps) {
  const int lane = threadIdx.x & 31;
  const float z[8] = {};
  for (int64_t q0 = wid * 32; q0 < p.R; q0 += warps * 32) {
    const int32_t s = q0 + lane < p.R ? p.src[q0 + lane] : 0;
    uint32_t none = __ballot_sync(0xFFFFFFFFu, s < 0 || s >= p.R);
    while (none) {
      const int64_t q = q0 + __ffs(none) - 1;
      none &= none - 1;
      for (int c = 8 * lane; c < int(p.D); c += 256) store8(p.rows_out + q * p.ld_rows_out + c, int(p.D) - c, z);
    }
  }
}

// Eight places of a token at a time: lane j holds the j-th, and the weight.
struct Places {
  int32_t slot;
  float w;
};
__device__ __forceinline__ Places places_of(const RowsP& p, int64_t t, int64_t k0, int lane) {
  Places v = {-1, 1.0f};
  if (lane < 8 && k0 + lane < p.K) {
    const int64_t j = t * p.K + k0 + lane;
    v.slot = p.slot[j];
    if (v.slot >= p.R) v.slot = -1;
    if (p.w) v.w = p.w[j];
  }
  return v;
}

// One warp per token and 256 C columns: its part of the row is read once, C
// loads at a time, and stored at each of the token's places.
template <int C>
__global__ void __launch_bounds__(kRowWarps * 32) dispatch_kernel(const RowsP p) {
  const int lane = threadIdx.x & 31;
  const int64_t wid = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5), warps = int64_t(gridDim.x) * kRowWarps;
  const int64_t parts = (p.D + 256 * C - 1) / (256 * C);
  after_previous();
  for (int64_t u = wid; u < p.T * parts; u += warps) {
    const int64_t t = u / parts;
    const int c0 = int(u % parts) * 256 * C + 8 * lane, D = int(p.D);
    uint4 v[C];
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (c0 + 256 * i < D) v[i] = raw8(p.tokens_in + t * p.ld_tokens + c0 + 256 * i, D - c0 - 256 * i);
    for (int64_t k0 = 0; k0 < p.K; k0 += 8) {
      const Places at = places_of(p, t, k0, lane);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int32_t q = __shfl_sync(0xFFFFFFFFu, at.slot, k);
        if (q < 0) continue;
        uint16_t* o = p.rows_out + q * p.ld_rows_out + c0;
#pragma unroll
        for (int i = 0; i < C; ++i)
          if (c0 + 256 * i < D) put8(o + 256 * i, D - c0 - 256 * i, v[i]);
      }
    }
  }
  zero_rows(p, wid, warps);
}

// One warp per token and 256 columns, eight rows' loads at a time.  The chunk in
// which the width ends is loaded whole too, here and below, except of the last
// row: the next one starts behind it.  (Loaded in pieces, put together before
// the next row's, 16384 x 8 rows of 2041 took 192 us here and 206 below.)
__global__ void __launch_bounds__(kRowWarps * 32) combine_kernel(const RowsP p) {
  const int lane = threadIdx.x & 31;
  const int64_t wid = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5), warps = int64_t(gridDim.x) * kRowWarps;
  const int64_t parts = (p.D + 255) / 256;
  const int32_t last = int32_t(p.R) - 1;
  after_previous();
  for (int64_t u = wid; u < p.T * parts; u += warps) {
    const int64_t t = u / parts;
    const int c = int(u % parts) * 256 + 8 * lane, left = int(p.D) - c;
    float v[8] = {};
    if (p.residual && left > 0) load8(p.residual + t * p.ld_residual + c, left, v);
    for (int64_t k0 = 0; k0 < p.K; k0 += 8) {
      const Places at = places_of(p, t, k0, lane);
      uint4 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int32_t q = __shfl_sync(0xFFFFFFFFu, at.slot, k);
        x[k] = q >= 0 && left > 0 ? raw8(p.rows_in + q * p.ld_rows + c, q < last ? 8 : left) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int32_t q = __shfl_sync(0xFFFFFFFFu, at.slot, k);
        const float w = __shfl_sync(0xFFFFFFFFu, at.w, k);
        if (q < 0) continue;  // its weight may be anything
        float f[8];
        unpack8(x[k], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fmaf(w, f[i], v[i]);
      }
    }
    if (left > 0) store8(p.tokens_out + t * p.ld_tokens + c, left, v);
  }
}

// One warp per token: dout's row goes out, weighted, to each of its places,
// and its product with the row there is the weight's gradient.  Eight rows'
// loads at a time; dout is read once per eight choices.
__global__ void __launch_bounds__(kRowWarps * 32) combine_bwd_kernel(const RowsP p) {
  const int lane = threadIdx.x & 31;
  const int64_t wid = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5), warps = int64_t(gridDim.x) * kRowWarps;
  const int32_t last = int32_t(p.R) - 1;
  after_previous();
  for (int64_t t = wid; t < p.T; t += warps)
    for (int64_t k0 = 0; k0 < p.K; k0 += 8) {
      const Places at = places_of(p, t, k0, lane);
      float dot[8] = {};
      for (int c0 = 0; c0 < int(p.D); c0 += 256) {
        const int c = c0 + 8 * lane, left = int(p.D) - c;  // left <= 0: this lane has none
        uint4 x[8];
        float d[8] = {};
        if (left > 0) load8(p.tokens_in + t * p.ld_tokens + c, left, d);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int32_t q = __shfl_sync(0xFFFFFFFFu, at.slot, k);
          x[k] = q >= 0 && left > 0 ? raw8(p.rows_in + q * p.ld_rows + c, q < last ? 8 : left) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int32_t q = __shfl_sync(0xFFFFFFFFu, at.slot, k);
          const float w = __shfl_sync(0xFFFFFFFFu, at.w, k);
          if (q < 0 || left <= 0) continue;
          float f[8];
          unpack8(x[k], f);
          if (left < 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = i < left ? f[i] : 0.0f;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[k] = fmaf(d[i], f[i], dot[k]);
            f[i] = w * d[i];
          }
          store8(p.rows_out + q * p.ld_rows_out + c, left, f);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float s = warp_sum(dot[k]);
        if (lane == 0 && k0 + k < p.K) p.dw[t * p.K + k0 + k] = s;
      }
    }
  zero_rows(p, wid, warps);
}

RowsP rows_of(const glu_block_rows_args& a) {
  RowsP p;
  p.T = a.T;
  p.K = a.K;
  p.D = a.D;
  p.R = a.T * a.K;
  p.ld_tokens = a.ld_tokens;
  p.ld_rows = a.ld_rows;
  p.ld_rows_out = a.ld_rows_out;
  p.ld_residual = a.ld_residual;
  p.slot = a.slot;
  p.src = a.src;
  p.w = a.w;
  p.tokens_in = static_cast<const uint16_t*>(a.tokens_in);
  p.rows_in = static_cast<const uint16_t*>(a.rows_in);
  p.residual = static_cast<const uint16_t*>(a.residual);
  p.tokens_out = static_cast<uint16_t*>(a.tokens_out);
  p.rows_out = static_cast<uint16_t*>(a.rows_out);
  p.dw = a.dw;
  return p;
}

int row_grid(int64_t warps, const DevInfo& d) {
  const int64_t blocks = (warps + kRowWarps - 1) / kRowWarps, most = int64_t(d.sms) * (64 / kRowWarps);
  return int(blocks < most ? blocks : most);
}

}  // namespace

size_t route_workspace(int64_t T, int64_t K, int32_t E) {
  const int64_t n = T * K, per = sort_per_block(n);
  return n <= per ? 0 : size_t((n + per - 1) / per) * size_t(E) * 4;
}

cudaError_t launch_route(const glu_block_route_args& a, cudaStream_t s) {
  RouteP p;
  p.ids = a.ids;
  p.slot = a.slot;
  p.src = a.src;
  p.offsets = a.offsets;
  p.hist = static_cast<int32_t*>(a.workspace);
  p.n = a.T * a.K;
  p.per_block = sort_per_block(p.n);
  p.E = a.E;
  p.id_bytes = a.id_bytes;
  p.blocks = int32_t((p.n + p.per_block - 1) / p.per_block);
  const int smem = kSortWarps * a.E * 4;
  static SmemLimit limit;
  cudaError_t e = limit.raise(reinterpret_cast<const void*>(route_place_kernel), kSortWarps * kMaxExperts * 4);
  if (e != cudaSuccess) return e;
  if (p.blocks > 1) e = launch_kernel(route_count_kernel, p.blocks, kSortThreads, 0, s, p, true);
  if (e != cudaSuccess) return e;
  return launch_kernel(route_place_kernel, p.blocks, kSortThreads, smem, s, p, true);
}

cudaError_t launch_dispatch(const glu_block_rows_args& a, cudaStream_t s, const DevInfo& d) {
  const RowsP p = rows_of(a);
  // 1024 columns per warp (four loads in flight) where there are enough
  // tokens to fill the SMs that way
  if (p.T * ((p.D + 1023) / 1024) >= int64_t(d.sms) * 32)
    return launch_kernel(dispatch_kernel<4>, row_grid(p.T * ((p.D + 1023) / 1024), d), kRowWarps * 32, 0, s, p, true);
  return launch_kernel(dispatch_kernel<1>, row_grid(p.T * ((p.D + 255) / 256), d), kRowWarps * 32, 0, s, p, true);
}

cudaError_t launch_combine(const glu_block_rows_args& a, cudaStream_t s, const DevInfo& d) {
  const RowsP p = rows_of(a);
  return launch_kernel(combine_kernel, row_grid(p.T * ((p.D + 255) / 256), d), kRowWarps * 32, 0, s, p, true);
}

cudaError_t launch_combine_bwd(const glu_block_rows_args& a, cudaStream_t s, const DevInfo& d) {
  const RowsP p = rows_of(a);
  return launch_kernel(combine_bwd_kernel, row_grid(p.T > p.R / 32 ? p.T : p.R / 32, d), kRowWarps * 32, 0, s, p, true);
}

}  // namespace gq
