// Tiles of 256 rows by up to 256 columns for pairs of CTAs, dense or by expert, and
// how many pairs run at once: what the linear layers' kernels share.
#pragma once

#include <atomic>

#include "block.h"
#include "block_util.cuh"

namespace gq {

constexpr int kTile = 256;        // rows of D per pair, and most columns
constexpr int kHalf = kTile / 2;  // rows of A and most columns of B per CTA
constexpr int kStep = 32;         // granularity of a tile's columns

enum Product { kForward, kGradX, kGradW };

// The functions take a kernel's parameters as P: offsets (NULL: dense), E experts
// (dense: 1), rows of x and dy, cols of a dw, n_at tiles of rows of D, `most`
// tokens of a tile, depth of the sum and the parts (splits) that it is cut into,
// whole slices of BK.
struct TilePlan {
  int32_t cut[kMaxExperts + 1];    // first row of each expert, in range and not falling
  int32_t order[kMaxExperts];      // experts by falling row count
  int32_t first[kMaxExperts + 1];  // tiles before each expert's, in that order
};

struct Tile {
  int32_t e, a0;           // expert; first row of D
  int32_t b0, b_end;       // columns of D: tokens, or columns of a dw
  int32_t n;               // columns computed (b_end - b0 rounded up)
  int32_t k0, k_end;       // summed range
  int32_t k_main;          // where the ring's part of it ends (dw: whole sixteens)
  int32_t split;           // the part of the sum that the range is
};

// `rows` tokens in equal tiles of at most `most`.
__device__ __forceinline__ int32_t token_tiles(int32_t rows, int32_t most) { return (rows + most - 1) / most; }

// Tile t of the walk: bands of eight row tiles of D, the columns inside, so
// that the pairs at work share a band's rows of A and a few columns of B in
// L2.
template <int PROD, int BK, typename P>
__device__ __forceinline__ Tile tile_at(const P& p, const TilePlan& plan, int32_t t) {
  Tile x;
  x.e = x.split = 0;
  if (PROD != kGradW && p.splits > 1) {
    x.split = t % p.splits;
    t /= p.splits;
  }
  int32_t rows0 = 0, rows1 = p.rows;
  if (p.offsets) {
    int32_t lo = 0, hi = p.E - 1;  // last one in order whose first tile is not after t
    while (lo < hi) {
      const int32_t mid = (lo + hi + 1) >> 1;
      if (plan.first[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    t -= plan.first[lo];
    x.e = plan.order[lo];
    rows0 = plan.cut[x.e];
    rows1 = plan.cut[x.e + 1];
  }
  const int32_t n_bt = PROD == kGradW ? (p.cols + kTile - 1) / kTile : token_tiles(rows1 - rows0, p.most);
  constexpr int32_t kBand = 8;
  const int32_t band = t / (kBand * n_bt), rem = t - band * kBand * n_bt;
  const int32_t high = min(kBand, p.n_at - band * kBand);
  const int32_t bt = rem / high, at = band * kBand + rem % high;
  x.a0 = at * kTile;
  if (PROD == kGradW) {
    x.b0 = bt * kTile;
    x.b_end = p.cols;
    x.n = kTile;
    x.k0 = rows0;
    x.k_end = rows1;
  } else {
    const int32_t each = ((rows1 - rows0 + n_bt - 1) / n_bt + kStep - 1) / kStep * kStep;
    x.b0 = rows0 + bt * each;
    x.b_end = min(rows1, x.b0 + each);
    x.n = min(each, (x.b_end - x.b0 + kStep - 1) / kStep * kStep);
    x.k0 = 0;
    x.k_end = p.depth;
    if (p.splits > 1) {  // whole slices, as equal as they go
      const int32_t slices = (p.depth + BK - 1) / BK;
      x.k0 = slices * x.split / p.splits * BK;
      x.k_end = min(p.depth, slices * (x.split + 1) / p.splits * BK);
    }
  }
  x.k_main = PROD == kGradW ? x.k_end - (x.k_end - x.k0) % 16 : x.k_end;
  return x;
}

// The experts' row ranges, their order and tile counts, by the whole block.
// The tiles go round the pairs, those of the largest expert first.  A dw's tiles
// are as large as their expert's rows, so they fall and the pairs' sums differ by
// no more than one tile.  For y and dx an expert's last token tile is smaller than
// its others, and some pairs may get more of the one kind (152 experts of 257 rows
// with two row tiles each: 1280 tokens for half of the 76 pairs, 1024 for the
// others).  Beyond 256 experts, where ranking them would take longer than it is
// worth, they go in their own order.
template <int PROD, typename P>
__device__ __forceinline__ void plan_tiles(const P& p, TilePlan& plan, int warp, int lane) {
  const int32_t col_tiles = (p.cols + kTile - 1) / kTile;
  if (!p.offsets) {
    if (threadIdx.x == 0) plan.first[1] = p.n_at * (PROD == kGradW ? col_tiles : token_tiles(p.rows, p.most) * p.splits);
    return;
  }
  if (warp == 0) {
    int32_t row = 0;
    for (int32_t e0 = 0; e0 < p.E; e0 += 32) {
      const int32_t e = e0 + lane;
      // ends in range, and a running maximum so that none falls
      int32_t end = e < p.E ? max(0, min(p.offsets[e + 1], p.rows)) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t u = __shfl_up_sync(0xFFFFFFFFu, end, o);
        if (lane >= o) end = max(end, u);
      }
      end = max(end, row);
      if (e < p.E) {
        plan.cut[e + 1] = end;
        plan.order[e] = e;
      }
      row = __shfl_sync(0xFFFFFFFFu, end, 31);
    }
    if (lane == 0) plan.cut[0] = 0;
  }
  __syncthreads();
  if (p.E <= 256) {
    for (int32_t e = threadIdx.x; e < p.E; e += blockDim.x) {
      const int32_t own = plan.cut[e + 1] - plan.cut[e];
      int32_t rank = 0;
      for (int32_t f = 0; f < p.E; ++f) {
        const int32_t n = plan.cut[f + 1] - plan.cut[f];
        rank += n > own || (n == own && f < e);
      }
      plan.order[rank] = e;
    }
    __syncthreads();
  }
  if (warp == 0) {
    int32_t tiles = 0;
    for (int32_t i0 = 0; i0 < p.E; i0 += 32) {
      const int32_t i = i0 + lane, e = i < p.E ? plan.order[i] : 0;
      const int32_t own = i >= p.E ? 0 : p.n_at * (PROD == kGradW ? col_tiles : token_tiles(plan.cut[e + 1] - plan.cut[e], p.most));
      int32_t n = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t u = __shfl_up_sync(0xFFFFFFFFu, n, o);
        if (lane >= o) n += u;
      }
      if (i < p.E) plan.first[i] = tiles + n - own;
      tiles += __shfl_sync(0xFFFFFFFFu, n, 31);
    }
    if (lane == 0) plan.first[p.E] = tiles;
  }
}

// Pairs that the current device runs at once: fewer than half its SMs where a
// GPC's SMs do not all pair up, and a pair more than that would run as a
// second wave.  Asked once per device and
// kept in `known` (devices are never reconfigured).
inline cudaError_t pairs_at_once(std::atomic<int> (&known)[64], const void* kern, int threads, int smem, const DevInfo& d, int* pairs) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  *pairs = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (*pairs > 0) return cudaSuccess;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(d.sms / 2 * 2));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(pairs, kern, &cfg);
  if (e != cudaSuccess) return e;
  if (*pairs < 1) return cudaErrorLaunchOutOfResources;
  if (dev < 64) known[dev].store(*pairs, std::memory_order_relaxed);
  return cudaSuccess;
}

}  // namespace gq
