// Linear layers, dense or by expert, forward and backward (glu_block.h), on
// the tcgen05 tensor cores:
//
//   y  = act(x W^T + b) + residual   summed over K
//   dx = dz W                        summed over N
//   dw = dz^T x                      summed over the tokens
//
// One kernel computes D[i, j] = sum_k A[i, k] B[j, k] for the three, in tiles
// of 256 rows by up to 256 columns, each by a pair of CTAs (cta_group::2): a
// CTA loads 128 rows of A and half of B's columns, and holds the accumulators
// of its own rows.  So each SM moves 32 KB per 64-wide slice of the sum instead
// of the 48 KB of a 128 x 256 tile of its own, and a ring of six stages fits.
//
// For y and dx, A is the weight and B the tokens, i.e. the tile is computed
// transposed: the tokens are then the dimension whose size the instruction
// leaves free (32 to 256 in steps of 32), and an expert's last rows cost what
// they are, not a whole tile.  The accumulator's rows come back with one
// output column per thread; quads of lanes swap 4 x 4 blocks so that each
// stores four consecutive ones.  For dw, A is dz and B is x.
//
// An operand whose contiguous dimension is the summed one (x and W forward, dz
// for dx) is loaded as a K-major tile, the others (W for dx, dz and x for
// dw) as M/N-major ones: TMA fetches boxes of 64 contiguous elements by rows
// in both cases, and the matrix descriptors say which way they run, so
// nothing is transposed in memory.
//
// By expert the rows are cut at offsets[e]: a tile of y or dx has tokens of
// one expert (those of the next one that its boxes also fetched are not
// stored); a tile of dw sums over one expert's rows, 16 at a time.  Its last
// rows, fewer than 16, come through a buffer of their own, ahead of the others,
// where the rows of the next expert are zeroed (so that what they hold, NaN
// included, does not count) while the sum over the whole sixteens goes on.
// (Zeroed in the ring's stages they held the products up: 242 us against 197
// for 64 uneven experts of 32768 x 2048 x 2048, then; 204 to 207 now.)
//
// Ten warps per CTA (dw: eleven, one for those last rows): one issues the loads,
// one (of CTA 0) the products into one of two accumulators in tensor memory,
// eight read the other accumulator and store it (sixteen were no faster: 278
// against 273 us at 4096 x 8192 x 7168, the issuing warps wait longer for their
// turn).  The two issuing warps run uniformly and elect a lane, so that operands
// and addresses stay in uniform registers: 274 to 253 us there (1900 TFLOP/s, as
// cuBLAS).  Where there are few tiles it is behind that: 7168 x 8192 takes 26 us
// for 32 tokens and 72 for 1024 (cuBLAS 21 and 61), the dw of 1024 x 1024 and 4096
// tokens, 16 tiles for 76 pairs, 22 us (8.5).  Every wait is bounded.
#include <atomic>
#include <cstring>

#include "block.h"
#include "block_act.cuh"
#include "block_linear.cuh"
#include "block_util.cuh"
#include "tc.cuh"
#include "tma.cuh"

namespace gq {
namespace {

constexpr int kTile = 256;           // rows of D per pair, and most columns
constexpr int kHalf = kTile / 2;     // rows of A and most columns of B per CTA
constexpr int kBK = 64, kStages = 6;
constexpr int kOperand = kHalf * kBK * 2;  // 16 KB
constexpr int kStageBytes = 2 * kOperand;
constexpr int kBox = 64 * kBK * 2;   // one M/N-major box: 64 elements by 64 k
constexpr int kTailBox = 64 * 16 * 2;                      // the same by 16 k
constexpr int kTailBytes = 2 * (kHalf / 64) * kTailBox;    // A's and B's boxes of a CTA
constexpr int kStep = 32;            // granularity of a tile's columns
constexpr int kEpiWarps = 8;
// warps: loads, products, epilogue, and for dw one for the last rows
constexpr int threads_of(bool dw) { return (2 + kEpiWarps + (dw ? 1 : 0)) * 32; }
constexpr uint32_t kTmemCols = 2 * kTile;
constexpr uint32_t kIdescK = tc::idesc_bf16_f32(kTile, 0);  // the columns are added per tile

enum Product { kForward, kGradX, kGradW };

struct Ctl {
  uint64_t full[kStages];   // CTA 0's: its arrival and the bytes of both CTAs
  uint64_t empty[kStages];  // each CTA's own: the products on its stage are done
  uint64_t tfull[2];        // each CTA's own: the accumulator is complete
  uint64_t tempty[2];       // each CTA's own: its warps have read it; CTA 0's: so have CTA 1's
  // dw, two buffers of last rows: landed (each CTA's own), cut short in both
  // CTAs (CTA 0's), multiplied (each CTA's own)
  uint64_t tail_full[2], tail_ready[2], tail_free[2];
  uint64_t done;            // each CTA's own: all products are done
  uint32_t tmem;
  int32_t cut[kMaxExperts + 1];    // first row of each expert, in range and not falling
  int32_t order[kMaxExperts];      // experts by falling row count
  int32_t first[kMaxExperts + 1];  // tiles before each expert's, in that order
};
constexpr int kSmem = 1024 + kStages * kStageBytes + 2 * kTailBytes + int(sizeof(Ctl));
static_assert(kSmem <= 232448, "shared memory per CTA exceeds 227 KB");

__device__ uint32_t g_err_linear;

struct LinearP {
  // tb[i]: boxes of 128 >> i rows, for tiles with fewer columns; dw: tb[0], and
  // ta16, tb[1] by 16 rows
  CUtensorMap ta, tb[3], ta16;
  const int32_t* offsets;    // NULL: dense
  int32_t E;                 // experts (dense: 1)
  int32_t rows;              // of x and dy
  int32_t width;             // rows of D: N, K (kGradX) or N
  int32_t cols;              // columns of D of a dw (K)
  int32_t depth;             // summed over (kForward: K, kGradX: N)
  int32_t n_at;              // tiles of 256 rows of D
  int32_t most;              // most tokens of a tile (a multiple of 32, up to 256)
  int64_t ld_out, stride_out, ld_residual, ld_z;
  uint16_t *out, *z;
  const uint16_t* residual;
  const void* bias;
  int32_t b32;
  int32_t splits;   // parts of the sum (dense y and dx of few tokens): fp32 parts to `part`
  float* part;      // [splits, rows, ld_part]
  int64_t ld_part;
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
template <int PROD>
__device__ __forceinline__ Tile tile_at(const LinearP& p, const Ctl* ctl, int32_t t) {
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
      if (ctl->first[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    t -= ctl->first[lo];
    x.e = ctl->order[lo];
    rows0 = ctl->cut[x.e];
    rows1 = ctl->cut[x.e + 1];
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
      const int32_t slices = (p.depth + kBK - 1) / kBK;
      x.k0 = slices * x.split / p.splits * kBK;
      x.k_end = min(p.depth, slices * (x.split + 1) / p.splits * kBK);
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
template <int PROD>
__device__ __forceinline__ void plan_tiles(const LinearP& p, Ctl* ctl, int warp, int lane) {
  const int32_t col_tiles = (p.cols + kTile - 1) / kTile;
  if (!p.offsets) {
    if (threadIdx.x == 0) ctl->first[1] = p.n_at * (PROD == kGradW ? col_tiles : token_tiles(p.rows, p.most) * p.splits);
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
        ctl->cut[e + 1] = end;
        ctl->order[e] = e;
      }
      row = __shfl_sync(0xFFFFFFFFu, end, 31);
    }
    if (lane == 0) ctl->cut[0] = 0;
  }
  __syncthreads();
  if (p.E <= 256) {
    for (int32_t e = threadIdx.x; e < p.E; e += blockDim.x) {
      const int32_t own = ctl->cut[e + 1] - ctl->cut[e];
      int32_t rank = 0;
      for (int32_t f = 0; f < p.E; ++f) {
        const int32_t n = ctl->cut[f + 1] - ctl->cut[f];
        rank += n > own || (n == own && f < e);
      }
      ctl->order[rank] = e;
    }
    __syncthreads();
  }
  if (warp == 0) {
    int32_t tiles = 0;
    for (int32_t i0 = 0; i0 < p.E; i0 += 32) {
      const int32_t i = i0 + lane, e = i < p.E ? ctl->order[i] : 0;
      const int32_t own = i >= p.E ? 0 : p.n_at * (PROD == kGradW ? col_tiles : token_tiles(ctl->cut[e + 1] - ctl->cut[e], p.most));
      int32_t n = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t u = __shfl_up_sync(0xFFFFFFFFu, n, o);
        if (lane >= o) n += u;
      }
      if (i < p.E) ctl->first[i] = tiles + n - own;
      tiles += __shfl_sync(0xFFFFFFFFu, n, 31);
    }
    if (lane == 0) ctl->first[p.E] = tiles;
  }
}

// Four 16-bit values per lane (two per word) of N independent 4 x 4 blocks,
// each held by a quad of lanes, transposed: value j of lane l becomes value l %
// 4 of lane j.  The blocks go through the exchanges together, so that their
// latencies overlap.
template <int N>
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[N][2], int lane) {
  const bool odd = lane & 1, up = lane & 2;
  uint32_t keep[N], got[N];
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const uint32_t even_half = __byte_perm(w[q][0], w[q][1], 0x5410), odd_half = __byte_perm(w[q][0], w[q][1], 0x7632);
    keep[q] = odd ? odd_half : even_half;
    got[q] = __shfl_xor_sync(0xFFFFFFFFu, odd ? even_half : odd_half, 1);
  }
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const uint32_t first = odd ? got[q] : keep[q], second = odd ? keep[q] : got[q];  // of the even and the odd lane
    const uint32_t a = __byte_perm(first, second, 0x5410), b = __byte_perm(first, second, 0x7632);
    keep[q] = up ? b : a;
    got[q] = __shfl_xor_sync(0xFFFFFFFFu, up ? a : b, 2);
  }
#pragma unroll
  for (int q = 0; q < N; ++q) {
    w[q][0] = up ? got[q] : keep[q];
    w[q][1] = up ? keep[q] : got[q];
  }
}

// Four consecutive bf16 of an output row (8-byte aligned), or its first n.
__device__ __forceinline__ void store4(uint16_t* o, int n, const uint32_t (&w)[2]) {
  if (n >= 4) {
    *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
  } else {
    if (n > 0) o[0] = uint16_t(w[0]);
    if (n > 1) o[1] = uint16_t(w[0] >> 16);
    if (n > 2) o[2] = uint16_t(w[1]);
  }
}

// Where a warp's 32 tokens of y, z or the residual begin: the lane's token of
// each quad, and its four columns.
struct TokenView {
  int32_t left;  // of the row from the lane's first column on
  int32_t rows;  // of the tokens from the lane's first one on
};
__device__ __forceinline__ void store_quads(uint16_t* o, int64_t ld, const TokenView& t, uint32_t (&w)[8][2], int lane) {
  quad_transpose(w, lane);
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (4 * q < t.rows) store4(o + 4 * q * ld, t.left, w[q]);
}
__device__ __forceinline__ void load_quads(const uint16_t* s, int64_t ld, const TokenView& t, uint32_t (&w)[8][2]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    w[q][0] = w[q][1] = 0;
    if (4 * q >= t.rows) continue;
    const uint16_t* v = s + 4 * q * ld;
    if (t.left >= 4) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(v));
      w[q][0] = x.x, w[q][1] = x.y;
    } else {
      if (t.left > 0) w[q][0] = v[0];
      if (t.left > 1) w[q][0] |= uint32_t(v[1]) << 16;
      if (t.left > 2) w[q][1] = v[2];
    }
  }
}

// The 4 x 4 block of 16-byte pieces that a quad of lanes holds (lane l: pieces
// 0 .. 3 of a row in w[0..3], w[4..7], ...) transposed: lane l then has piece l
// % 4 of the quad's four rows.
__device__ __forceinline__ void piece_transpose(uint32_t (&w)[16], int lane) {
  const bool odd = lane & 1, up = lane & 2;
#pragma unroll
  for (int i = 0; i < 8; ++i) {  // pieces 0, 1 and 2, 3 between neighbours
    const int lo = (i / 4) * 8 + i % 4, hi = lo + 4;
    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, odd ? w[lo] : w[hi], 1);
    if (odd) w[lo] = got;
    else w[hi] = got;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {  // pieces 0, 2 and 1, 3 between pairs
    const int lo = i, hi = i + 8;
    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? w[lo] : w[hi], 2);
    if (up) w[lo] = got;
    else w[hi] = got;
  }
}

template <int PROD, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads_of(PROD == kGradW), 1) linear_kernel(const __grid_constant__ LinearP p) {
  constexpr bool kAmn = PROD != kForward, kBmn = PROD == kGradW;
  constexpr uint32_t kIdesc = kIdescK | (kAmn ? 1u << 15 : 0u) | (kBmn ? 1u << 16 : 0u);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* tails = stages + kStages * kStageBytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(tails + 2 * kTailBytes);
  const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int32_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  after_previous();
  if (threadIdx.x == 32) {
    prefetch_tensormap(&p.ta);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl->tfull[b], 1);
      mbar_init(&ctl->tempty[b], rank == 0 ? kEpiWarps + 1 : kEpiWarps);
      mbar_init(&ctl->tail_full[b], 1);
      mbar_init(&ctl->tail_ready[b], 2);
      mbar_init(&ctl->tail_free[b], 1);
    }
    mbar_init(&ctl->done, 1);
    fence_barrier_init();
  }
  plan_tiles<PROD>(p, ctl, warp, lane);
  if (warp == 1) {
    __syncwarp();
    tc::pair_alloc(&ctl->tmem, kTmemCols);
    tc::pair_relinquish();
  }
  tc::fence_before();
  cluster_sync();
  tc::fence_after();
  const uint32_t tmem = ctl->tmem;
  const int32_t tiles = ctl->first[p.offsets ? p.E : 1];

  if (warp == 0) {
    // ---------------------------------------------------------- producer --
    // the warp runs as one, so that what it computes stays in uniform
    // registers; one lane issues
    int s = 0, held = 0;  // held: stages ever filled, up to all
    uint32_t parity = 0;
    uint32_t tail = 0;  // buffers of last rows filled
    const uint32_t full0 = peer_addr(&ctl->full[0], 0);
    bool ok = true;
    for (int32_t t = pair; t < tiles && ok; t += pairs) {
      const Tile x = tile_at<PROD>(p, ctl, t);
      const int32_t a0 = x.a0 + int32_t(rank) * kHalf, half = x.n / 2, b0 = x.b0 + int32_t(rank) * half;
      // the smallest box with the half's columns (more than it needs are not
      // multiplied)
      const int box = half > 64 ? 0 : half > 32 ? 1 : 2;
      const uint32_t bytes = uint32_t(kOperand + (kHalf >> box) * kBK * 2);
      const CUtensorMap* tb = &p.tb[PROD == kGradW ? 0 : box];
      if (PROD == kGradW && x.k_main < x.k_end) {
        const int u = int(tail & 1u);
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->tail_free[u], ((tail >> 1) & 1u) ^ 1u));
        if (!ok) {
          if (lane == 0) atomicOr(&g_err_linear, kErrWaitEmpty);
          break;
        }
        if (tc::elect_one()) {
          uint8_t* a = tails + u * kTailBytes;
          const uint32_t bar = smem_u32(&ctl->tail_full[u]);
          mbar_arrive_expect_tx(&ctl->tail_full[u], kTailBytes);
#pragma unroll
          for (int i = 0; i < kHalf / 64; ++i) {
            pair_load_2d(a + i * kTailBox, &p.ta16, a0 + 64 * i, x.k_main, bar);
            pair_load_2d(a + (kHalf / 64 + i) * kTailBox, &p.tb[1], b0 + 64 * i, x.k_main, bar);
          }
        }
        ++tail;
      }
      for (int32_t k = x.k0; k < x.k_main; k += kBK) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->empty[s], parity ^ 1u));
        if (!ok) {
          if (lane == 0) atomicOr(&g_err_linear, kErrWaitEmpty);
          break;
        }
        if (tc::elect_one()) {
          uint8_t* a = stages + s * kStageBytes;
          uint8_t* b = a + kOperand;
          const uint32_t bar = full0 + 8u * uint32_t(s);
          if (rank == 0) mbar_arrive_expect_tx(&ctl->full[s], 2 * bytes);
          if (PROD == kForward) {
            pair_load_3d(a, &p.ta, k, a0, x.e, bar);
          } else if (PROD == kGradX) {
#pragma unroll
            for (int i = 0; i < kHalf / 64; ++i) pair_load_3d(a + i * kBox, &p.ta, a0 + 64 * i, k, x.e, bar);
          } else {
#pragma unroll
            for (int i = 0; i < kHalf / 64; ++i) pair_load_2d(a + i * kBox, &p.ta, a0 + 64 * i, k, bar);
          }
          if (PROD == kGradW) {
#pragma unroll
            for (int i = 0; i < kHalf / 64; ++i) pair_load_2d(b + i * kBox, tb, b0 + 64 * i, k, bar);
          } else {
            pair_load_2d(b, tb, k, b0, bar);
          }
        }
        held = max(held, s + 1);
        if (++s == kStages) s = 0, parity ^= 1u;
      }
    }
    // never leave with loads in flight: the products on each stage's last slice
    // (which waited for its loads) are done
    if (s == held) s = 0, parity ^= 1u;
    for (int j = 0; j < held; ++j) {
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&ctl->empty[s], parity ^ 1u)) && lane == 0) atomicOr(&g_err_linear, kErrDrain);
      if (++s == held) s = 0, parity ^= 1u;
    }
    for (uint32_t j = tail > 2 ? tail - 2 : 0; j < tail; ++j)
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&ctl->tail_free[j & 1u], (j >> 1) & 1u)) && lane == 0) atomicOr(&g_err_linear, kErrDrain);
  } else if (warp == 1) {
    // --------------------------------------------------------------- MMA --
    int s = 0;
    uint32_t parity = 0;
    int32_t i = 0;
    const uint32_t a_addr = smem_u32(stages);
    const uint64_t ad0 = kAmn ? tc::sw128_mnmajor_desc(a_addr, kBox) : tc::sw128_kmajor_desc(a_addr);
    const uint64_t bd0 = kBmn ? tc::sw128_mnmajor_desc(a_addr + kOperand, kBox) : tc::sw128_kmajor_desc(a_addr + kOperand);
    uint32_t tail = 0;  // buffers of last rows multiplied
    bool ok = true;
    for (int32_t t = pair; t < tiles && ok && rank == 0; t += pairs) {
      const Tile x = tile_at<PROD>(p, ctl, t);
      if (x.k0 == x.k_end) continue;  // an expert without rows: the epilogue stores zeros
      const int b = i & 1;
      const uint32_t d = tmem + uint32_t(b * kTile);
      const uint32_t idesc = kIdesc | (uint32_t(x.n >> 3) << 17);
      ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(&ctl->tempty[b], ((uint32_t(i) >> 1) & 1u) ^ 1u));
      if (!ok && lane == 0) atomicOr(&g_err_linear, kErrWaitEmpty);
      tc::fence_after();
      for (int32_t k = x.k0; k < x.k_main && ok; k += kBK) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->full[s], parity));
        if (!ok) {
          if (lane == 0) atomicOr(&g_err_linear, kErrWaitFull);
          break;
        }
        tc::fence_after();
        if (tc::elect_one()) {
          const uint64_t ad = ad0 + uint32_t(s * (kStageBytes >> 4)), bd = bd0 + uint32_t(s * (kStageBytes >> 4));
#pragma unroll
          for (int j = 0; j < kBK / 16; ++j)
            if (PROD != kGradW || k + 16 * j < x.k_main)  // dw: 16 rows at a time, as far as there are some
              tc::pair_mma_bf16(d, ad + j * (kAmn ? 128 : 2), bd + j * (kBmn ? 128 : 2), idesc, uint32_t((k - x.k0) | j));
          tc::pair_commit(&ctl->empty[s]);
        }
        if (++s == kStages) s = 0, parity ^= 1u;
      }
      if (PROD == kGradW && ok && x.k_main < x.k_end) {
        const int u = int(tail & 1u);
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(&ctl->tail_ready[u], (tail >> 1) & 1u));
        if (!ok && lane == 0) atomicOr(&g_err_linear, kErrWaitFull);
        ++tail;
        tc::fence_after();
        if (ok && tc::elect_one()) {
          const uint32_t at = smem_u32(tails) + uint32_t(u * kTailBytes);
          tc::pair_mma_bf16(d, tc::sw128_mnmajor_desc(at, kTailBox), tc::sw128_mnmajor_desc(at + (kHalf / 64) * kTailBox, kTailBox), idesc,
                            uint32_t(x.k_main - x.k0));
          tc::pair_commit(&ctl->tail_free[u]);
        }
      }
      __syncwarp();
      if (ok && tc::elect_one()) tc::pair_commit(&ctl->tfull[b]);
      ++i;
    }
    // CTA 1's warp hands its CTA's reads of an accumulator on to CTA 0.  An arrival
    // there has to be a release at cluster scope, which waits for what its thread
    // has in flight: this warp has nothing, the epilogue's would wait for their
    // stores (64 even experts' dw 217 us, this way 195).
    for (int32_t t = pair; t < tiles && rank == 1; t += pairs) {
      const Tile x = tile_at<PROD>(p, ctl, t);
      if (x.k0 == x.k_end) continue;
      const int b = i & 1;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&ctl->tempty[b], (uint32_t(i) >> 1) & 1u))) {
        if (lane == 0) atomicOr(&g_err_linear, kErrWaitFull);
        break;
      }
      tc::fence_after();
      tc::fence_before();
      if (lane == 0) peer_arrive(peer_addr(&ctl->tempty[b], 0));
      ++i;
    }
    __syncwarp();
    if (tc::elect_one()) {  // the lane that issued the products
      if (rank == 0) tc::pair_commit(&ctl->done);
      if (!mbar_wait(&ctl->done, 0)) atomicOr(&g_err_linear, kErrDrain);
    }
    __syncwarp();
  } else if (warp == 2 + kEpiWarps) {
    // ------------------------------------------------------- dw: last rows --
    // zeroes the next expert's rows of the 16: whole 128-byte rows of every box
    // (the swizzle moves 16-byte pieces inside a row only)
    uint32_t tail = 0;
    for (int32_t t = pair; t < tiles; t += pairs) {
      const Tile x = tile_at<PROD>(p, ctl, t);
      const int32_t have = x.k_end - x.k_main;
      if (have == 0) continue;
      const int u = int(tail & 1u);
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&ctl->tail_full[u], (tail >> 1) & 1u))) {
        if (lane == 0) atomicOr(&g_err_linear, kErrWaitFull);
        break;
      }
      ++tail;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      const int32_t n = (16 - have) * 8;  // 16-byte pieces per box
      for (int32_t q = lane; q < n * (kTailBytes / kTailBox); q += 32)
        *reinterpret_cast<uint4*>(tails + u * kTailBytes + (q / n) * kTailBox + have * 128 + (q % n) * 16) = zero;
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) peer_arrive(peer_addr(&ctl->tail_ready[u], 0));
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- epilogue --
    const int quarter = warp & 3, group = (warp - 2) >> 2;
    int32_t i = 0;
    for (int32_t t = pair; t < tiles; t += pairs) {
      const Tile x = tile_at<PROD>(p, ctl, t);
      const int b = i & 1;
      if (x.k0 < x.k_end) {
        bool ok = true;
        if (lane == 0) {
          ok = mbar_wait(&ctl->tfull[b], (uint32_t(i) >> 1) & 1u);
          if (!ok) atomicOr(&g_err_linear, kErrWaitFull);
        }
        if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) break;
        tc::fence_after();
        ++i;
      }
      const int32_t row0 = x.a0 + int32_t(rank) * kHalf + quarter * 32;  // of D: this warp's 32
      const uint32_t tbase = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(b * kTile);
      float bias = 0.0f;
      if (PROD == kForward && p.bias && row0 + lane < p.width) {
        const int64_t at = int64_t(x.e) * p.width + row0 + lane;
        bias = p.b32 ? __ldg(static_cast<const float*>(p.bias) + at) : bf16_of_bits(__ldg(static_cast<const uint16_t*>(p.bias) + at));
      }
#pragma unroll 1
      for (int c = group * 32; c < x.n; c += 8 * kEpiWarps) {
        uint32_t r[32];
        // y and dx: this lane has column row0 + lane of 32 tokens in r, and
        // after the transposition four columns of every fourth token
        const int32_t token = x.b0 + c + (lane & 3), col = row0 + (lane & ~3);
        const TokenView view = {p.width - col, x.b_end - token};
        uint32_t res[8][2];
        if (PROD == kForward && p.residual && p.splits == 1)
          load_quads(p.residual + int64_t(token) * p.ld_residual + col, p.ld_residual, view, res);
        if (x.k0 < x.k_end) {
          tc::ld32(tbase + uint32_t(c), r);
          tc::wait_ld();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0;
        }
        if (PROD != kGradW && p.splits > 1) {
          float* part = p.part + (int64_t(x.split) * p.rows + x.b0 + c) * p.ld_part + row0 + lane;
          if (row0 + lane < p.width) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (x.b0 + c + j < x.b_end) part[j * p.ld_part] = __uint_as_float(r[j]);
          }
        } else if (PROD != kGradW) {
          uint32_t w[8][2];
          if (PROD == kForward) {
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + bias);
            if (p.z) {
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                w[q][0] = bf16x2_of(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]));
                w[q][1] = bf16x2_of(__uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3]));
              }
              store_quads(p.z + int64_t(token) * p.ld_z + col, p.ld_z, view, w, lane);
            }
            if (ACT != GLU_ACT_IDENTITY) {
#pragma unroll
              for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(act_value<ACT>(__uint_as_float(r[j])));
            }
            if (p.residual) {
              quad_transpose(res, lane);
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const uint32_t v = res[j / 4][(j / 2) & 1];
                r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float((j & 1) ? (v & 0xFFFF0000u) : (v << 16)));
              }
            }
          }
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            w[q][0] = bf16x2_of(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]));
            w[q][1] = bf16x2_of(__uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3]));
          }
          store_quads(p.out + int64_t(token) * p.ld_out + col, p.ld_out, view, w, lane);
        } else {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) w[j] = bf16x2_of(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
          piece_transpose(w, lane);
          const int32_t row = row0 + (lane & ~3), left = x.b_end - x.b0 - c - 8 * (lane & 3);
          uint16_t* out = p.out + x.e * p.stride_out + int64_t(row) * p.ld_out + x.b0 + c + 8 * (lane & 3);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (row + j >= p.width || left <= 0) continue;
            // stores that stay in L2 (streamed ones: 200 against 195 us for 64 uneven experts)
            const uint4 v = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
            if (left >= 8) *reinterpret_cast<uint4*>(out + j * p.ld_out) = v;
            else put8(out + j * p.ld_out, left, v);
          }
        }
      }
      if (x.k0 < x.k_end) {
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->tempty[b]);
      }
    }
    // rows that no expert has
    if (PROD != kGradW && p.offsets) {
      const float zero[8] = {};
      const int64_t chunks = (p.width + 7) / 8, first = ctl->cut[p.E];
      for (int64_t q = int64_t(blockIdx.x) * kEpiWarps * 32 + threadIdx.x - 64; q < (p.rows - first) * chunks;
           q += int64_t(gridDim.x) * kEpiWarps * 32) {
        const int64_t m = first + q / chunks;
        const int32_t c = int32_t(q % chunks) * 8;
        store8(p.out + m * p.ld_out + c, p.width - c, zero);
        if (PROD == kForward && p.z) store8(p.z + m * p.ld_z + c, p.width - c, zero);
      }
    }
  }
  __syncwarp();
  tc::fence_before();
  cluster_sync();
  if (warp == 1) {
    tc::fence_after();
    tc::pair_dealloc(tmem, kTmemCols);
  }
}

// Pairs that the current device runs at once: fewer than half its SMs where a
// GPC's SMs do not all pair up, and a pair more than that would run as a
// second wave.  Asked once per device (devices are never reconfigured).
cudaError_t pairs_at_once(const void* kern, int threads, const DevInfo& d, int* pairs) {
  static std::atomic<int> known[64];  // shared memory, one block per SM, limits every product alike
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
  cfg.dynamicSmemBytes = kSmem;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(pairs, kern, &cfg);
  if (e != cudaSuccess) return e;
  if (*pairs < 1) return cudaErrorLaunchOutOfResources;
  if (dev < 64) known[dev].store(*pairs, std::memory_order_relaxed);
  return cudaSuccess;
}

template <int PROD, int ACT>
cudaError_t launch_t(LinearP& p, cudaStream_t s, const DevInfo& d) {
  auto kern = linear_kernel<PROD, ACT>;
  static SmemLimit limit;
  cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern), kSmem);
  if (e != cudaSuccess) return e;
  p.n_at = (p.width + kTile - 1) / kTile;
  // by expert the device counts the tiles: no more than one token tile per
  // expert above the dense count
  const int64_t most = PROD == kGradW ? int64_t(p.n_at) * ((p.cols + kTile - 1) / kTile) * p.E
                                      : p.n_at * ((int64_t(p.rows) + p.most - 1) / p.most + (p.offsets ? p.E : 0)) * p.splits;
  int pairs = 0;
  e = pairs_at_once(reinterpret_cast<const void*>(kern), threads_of(PROD == kGradW), d, &pairs);
  if (e != cudaSuccess) return e;
  if (most < pairs) pairs = int(most);
  return launch_kernel(kern, 2 * pairs, threads_of(PROD == kGradW), kSmem, s, p, true);
}

// How the tokens of a dense y or dx are cut into tiles (at most `most` each)
// and the sum into parts, a function of the shape alone (76 pairs): the plan
// with the least estimated time.  A slice takes what its bytes take into the
// SM (16 KB of weights and 64 per token at about 115 KB per us, measured at
// 1024 x 7168 x 8192 with 128-wide tiles, 83 us, and 256-wide ones, 78 us), the
// busiest pair's tiles follow each other, and the join of split sums reads and
// writes the fp32 parts.
struct TokenPlan {
  int most, splits;
};
TokenPlan token_plan(int64_t rows, int64_t width, int64_t depth) {
  const int64_t at = (width + kTile - 1) / kTile, slices = (depth + kBK - 1) / kBK;
  TokenPlan best = {kTile, 1};
  double least = 1e30;
  for (int n = 1; n <= 8 && slices / n >= 8; ++n)
    for (int most = kTile; most >= 64; most -= kStep) {
      const int64_t bt = (rows + most - 1) / most, each = ((rows + bt - 1) / bt + kStep - 1) / kStep * kStep;
      double us = double((at * bt * n + 75) / 76) * (double((slices + n - 1) / n) * (16.384 + 0.064 * double(each)) / 115.0 + 0.5);
      if (n > 1) us += 3.0 + double(n) * double(rows) * double(width) * 8e-6 / 4.0;
      if (us < least * 0.98) least = us, best = {most, n};
    }
  return best;
}

int64_t padded8(int64_t n) { return (n + 7) / 8 * 8; }
int64_t dz_slots(const glu_block_linear_bwd_args& a) { return (a.M + kDzRows - 1) / kDzRows + (a.E > 0 ? a.E : 0); }
size_t dz_bytes(const glu_block_linear_bwd_args& a) {
  return a.act != GLU_ACT_IDENTITY && (a.dx || a.dw) ? size_t(a.M) * size_t(padded8(a.N)) * 2 : 0;
}

}  // namespace

static size_t part_bytes(int splits, int64_t rows, int64_t width) {
  return splits > 1 ? size_t(splits) * size_t(rows) * size_t(padded8(width)) * 4 : 0;
}
static TokenPlan fwd_plan(const glu_block_linear_fwd_args& a) {
  return a.E > 0 || linear_few(a) ? TokenPlan{kTile, 1} : token_plan(a.M, a.N, a.K);
}
static TokenPlan dx_plan(const glu_block_linear_bwd_args& a) {
  return a.E > 0 || !a.dx ? TokenPlan{kTile, 1} : token_plan(a.M, a.K, a.N);
}

size_t linear_fwd_workspace(const glu_block_linear_fwd_args& a) { return part_bytes(fwd_plan(a).splits, a.M, a.N); }
size_t linear_bwd_workspace(const glu_block_linear_bwd_args& a) {
  // dz, then the parts of db and those of dx, which follow each other on the stream
  const size_t db = a.db ? size_t(dz_slots(a)) * a.N * 4 : 0, dx = part_bytes(dx_plan(a).splits, a.M, a.K);
  return dz_bytes(a) + (db > dx ? db : dx);
}

// Maps of the tokens' rows (64-wide slices), in boxes of 128, 64 and 32 rows.
// Dense tiles are alike but for the last, which has no more columns: theirs and
// the narrower ones; by expert any.
static cudaError_t token_maps(LinearP& p, const void* t, int64_t cols, int64_t rows, int64_t ld, int most) {
  const int64_t tiles = (rows + most - 1) / most, half = ((rows + tiles - 1) / tiles + kStep - 1) / kStep * kStep / 2;
  cudaError_t e = cudaSuccess;
  for (int i = p.offsets || half > 64 ? 0 : half > 32 ? 1 : 2; i < 3 && e == cudaSuccess; ++i) {
    e = make_tile_map(&p.tb[i], t, 2, cols, rows, ld * 2, kBK, kHalf >> i, 128);
    if (!p.offsets && rows % (2 * half) == 0) break;  // no narrower last tile
  }
  return e;
}

cudaError_t launch_linear_fwd(const glu_block_linear_fwd_args& a, cudaStream_t s, const DevInfo& d) {
  if (linear_few(a)) return launch_linear_few(a, s);
  LinearP p;
  memset(&p, 0, sizeof p);
  const int64_t E = a.E > 0 ? a.E : 1;
  cudaError_t e = make_stack_map(&p.ta, a.w, a.K, a.N, a.ld_w * 2, E, (a.E > 0 ? a.stride_w : a.N * a.ld_w) * 2, kHalf);
  const TokenPlan plan = fwd_plan(a);
  p.offsets = a.E > 0 ? a.offsets : nullptr;
  if (e == cudaSuccess) e = token_maps(p, a.x, a.K, a.M, a.ld_x, plan.most);
  if (e != cudaSuccess) return e;
  p.E = int32_t(E);
  p.rows = int32_t(a.M);
  p.width = int32_t(a.N);
  p.depth = int32_t(a.K);
  p.splits = plan.splits;
  p.most = plan.most;
  p.part = static_cast<float*>(a.workspace);
  p.ld_part = padded8(a.N);
  p.out = static_cast<uint16_t*>(a.y);
  p.ld_out = a.ld_y;
  p.z = static_cast<uint16_t*>(a.z);
  p.ld_z = a.ld_z;
  p.residual = static_cast<const uint16_t*>(a.residual);
  p.ld_residual = a.ld_residual;
  p.bias = a.bias;
  p.b32 = a.b_fmt == GLU_FMT_FP32;
  if (p.splits > 1) {
    e = launch_t<kForward, GLU_ACT_IDENTITY>(p, s, d);
    return e == cudaSuccess ? launch_linear_join(a, p.part, p.splits, s) : e;
  }
  switch (a.act) {
    case GLU_ACT_SILU: return launch_t<kForward, GLU_ACT_SILU>(p, s, d);
    case GLU_ACT_GELU_TANH: return launch_t<kForward, GLU_ACT_GELU_TANH>(p, s, d);
    case GLU_ACT_RELU: return launch_t<kForward, GLU_ACT_RELU>(p, s, d);
    case GLU_ACT_GELU_ERF: return launch_t<kForward, GLU_ACT_GELU_ERF>(p, s, d);
    default: return launch_t<kForward, GLU_ACT_IDENTITY>(p, s, d);
  }
}

cudaError_t launch_linear_bwd(const glu_block_linear_bwd_args& a, cudaStream_t s, const DevInfo& d) {
  const int64_t E = a.E > 0 ? a.E : 1;
  const bool acts = a.act != GLU_ACT_IDENTITY;
  const void* dz = a.dy;
  int64_t ld_dz = a.ld_dy;
  cudaError_t e = cudaSuccess;
  if (a.db || (acts && (a.dx || a.dw))) {
    DzP q;
    q.dy = static_cast<const uint16_t*>(a.dy);
    q.z = static_cast<const uint16_t*>(a.z);
    q.dz = dz_bytes(a) ? static_cast<uint16_t*>(a.workspace) : nullptr;
    q.part = a.db ? reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + dz_bytes(a)) : nullptr;
    q.db = a.db;
    q.offsets = a.E > 0 ? a.offsets : nullptr;
    q.ld_dy = a.ld_dy;
    q.ld_z = a.ld_z;
    q.ld_dz = padded8(a.N);
    q.rows = int32_t(a.M);
    q.N = int32_t(a.N);
    q.E = int32_t(E);
    q.slots = int32_t(dz_slots(a));
    e = launch_linear_dz(a.act, q, s);
    if (e != cudaSuccess) return e;
    if (q.dz) dz = q.dz, ld_dz = q.ld_dz;
  }
  LinearP p;
  memset(&p, 0, sizeof p);
  p.offsets = a.E > 0 ? a.offsets : nullptr;
  p.E = int32_t(E);
  p.rows = int32_t(a.M);
  if (a.dx) {
    e = make_stack_map(&p.ta, a.w, a.K, a.N, a.ld_w * 2, E, (a.E > 0 ? a.stride_w : a.N * a.ld_w) * 2, kBK);
    const TokenPlan plan = dx_plan(a);
    if (e == cudaSuccess) e = token_maps(p, dz, a.N, a.M, ld_dz, plan.most);
    if (e != cudaSuccess) return e;
    p.width = int32_t(a.K);
    p.depth = int32_t(a.N);
    p.splits = plan.splits;
    p.most = plan.most;
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + dz_bytes(a));
    p.ld_part = padded8(a.K);
    p.out = static_cast<uint16_t*>(a.dx);
    p.ld_out = a.ld_dx;
    e = launch_t<kGradX, GLU_ACT_IDENTITY>(p, s, d);
    if (e == cudaSuccess && p.splits > 1) {
      glu_block_linear_fwd_args j = {};  // the join of a forward without bias, activation and residual
      j.act = GLU_ACT_IDENTITY;
      j.b_fmt = GLU_FMT_BF16;
      j.M = a.M;
      j.N = a.K;
      j.ld_y = a.ld_dx;
      j.y = a.dx;
      e = launch_linear_join(j, p.part, p.splits, s);
    }
    if (e != cudaSuccess) return e;
  }
  if (a.dw) {
    e = make_tile_map(&p.ta, dz, 2, a.N, a.M, ld_dz * 2, 64, kBK, 128);
    if (e == cudaSuccess) e = make_tile_map(&p.ta16, dz, 2, a.N, a.M, ld_dz * 2, 64, 16, 128);
    if (e == cudaSuccess) e = make_tile_map(&p.tb[0], a.x, 2, a.K, a.M, a.ld_x * 2, 64, kBK, 128);
    if (e == cudaSuccess) e = make_tile_map(&p.tb[1], a.x, 2, a.K, a.M, a.ld_x * 2, 64, 16, 128);
    if (e != cudaSuccess) return e;
    p.width = int32_t(a.N);
    p.cols = int32_t(a.K);
    p.out = static_cast<uint16_t*>(a.dw);
    p.ld_out = a.ld_dw;
    p.stride_out = a.stride_dw;
    p.splits = 1;
    p.most = kTile;
    e = launch_t<kGradW, GLU_ACT_IDENTITY>(p, s, d);
  }
  return e;
}

cudaError_t read_err_linear(uint32_t* v, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(v, g_err_linear, sizeof(uint32_t));
  if (e == cudaSuccess && clear) {
    const uint32_t z = 0;
    e = cudaMemcpyToSymbol(g_err_linear, &z, sizeof(uint32_t));
  }
  return e;
}

}  // namespace gq
