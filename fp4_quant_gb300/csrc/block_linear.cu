// Linear layers, dense or by expert, forward and backward (glu_block.h), on
// the tcgen05 tensor cores:
//
//   y  = act(x W^T + b) + residual   rows x columns = tokens x N, summed over K
//   dx = dz W                        tokens x K, summed over N
//   dw = dz^T x                      N x K, summed over the tokens
//
// One kernel computes D[i, j] = sum_k A[i, k] B[j, k] for the three.  An
// operand whose contiguous dimension is the summed one (x and W forward, dz
// for dx) is loaded as a K-major tile, the others (W for dx, dz and x for
// dw) as M/N-major ones: TMA fetches boxes of 64 contiguous elements by rows
// in both cases, and the matrix descriptors say which way they run, so
// nothing is transposed in memory.
//
// By expert the rows are cut at offsets[e]: a tile of dx or y has rows of one
// expert (those of the next one that its box also fetched are not stored), a
// tile of dw sums over one expert's rows (those of the next one are zeroed in
// shared memory before the product, so that what they hold, NaN included,
// does not count).
//
// Ten warps per block, as the gate/up GEMM: one issues the loads into a ring
// of stages, one the products into one of two accumulators in tensor memory,
// eight read the other accumulator and store it.  Every wait is bounded.
#include <cstring>

#include "block.h"
#include "block_util.cuh"
#include "tc.cuh"
#include "tma.cuh"

namespace gq {
namespace {

constexpr int kBM = 128, kBN = 256, kBK = 64, kStages = 4;
constexpr int kABytes = kBM * kBK * 2, kBBytes = kBN * kBK * 2, kStageBytes = kABytes + kBBytes;
constexpr int kBox = 64 * kBK * 2;  // one M/N-major box: 64 elements by 64 k
constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr uint32_t kTmemCols = 2 * kBN;
constexpr uint32_t kIdescK = tc::idesc_bf16_f32(kBM, kBN);

enum Product { kForward, kGradX, kGradW };

struct Ctl {
  uint64_t full[kStages], empty[kStages];
  uint64_t tfull[2], tempty[2];
  uint64_t done;
  uint32_t tmem;
  int32_t cut[kMaxExperts + 1];    // first row of each expert, in range and not falling
  int32_t first[kMaxExperts + 1];  // tiles before each expert's
};
constexpr int kSmem = 1024 + kStages * kStageBytes + int(sizeof(Ctl));
static_assert(kSmem <= 232448, "shared memory per CTA exceeds 227 KB");

__device__ uint32_t g_err_linear;

struct LinearP {
  CUtensorMap ta, tb;
  const int32_t* offsets;  // NULL: dense
  int32_t E;               // experts (dense: 1)
  int32_t rows;            // of x and dy
  int32_t M, N, K;         // the product's own: D [M, N] (kForward, kGradX: M = rows), sum over K (kGradW: rows)
  int32_t n_nt;            // column tiles of D
  int32_t n_mt;            // row tiles of D (kGradW; dense)
  int64_t ld_out, stride_out, ld_residual, ld_z;
  uint16_t *out, *z;
  const uint16_t* residual;
  const void* bias;
  int32_t b32, act;
};

// act(z), for values that are rounded to bf16 next.
__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case GLU_ACT_SILU: return __fdividef(z, 1.0f + __expf(-z));
    case GLU_ACT_GELU_TANH: {
      const float u = 1.5957691216057308f * fmaf(0.044715f * z * z, z, z);  // 2 sqrt(2 / pi) (z + 0.044715 z^3)
      return __fdividef(z, 1.0f + __expf(-u));                              // z sigmoid(u) = z (1 + tanh(u / 2)) / 2
    }
    case GLU_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case GLU_ACT_GELU_ERF: return z * normcdff(z);
    default: return z;
  }
}

struct Tile {
  int32_t e, m0, n0;       // expert; first row and column of D
  int32_t m_end;           // rows of D below this one are stored
  int32_t k0, k_end, nk;   // summed range and its 64-wide blocks
};

// Tile t of the walk.  Dense: bands of 16 row tiles, columns inside, so that
// the tiles at work share a band's rows of A and a few columns of B in L2.
template <int PROD>
__device__ __forceinline__ Tile tile_at(const LinearP& p, const Ctl* ctl, int32_t t) {
  Tile x;
  x.e = 0;
  int32_t lo = 0, rows0 = 0, rows1 = p.rows, n_mt = p.n_mt;
  if (p.offsets) {
    int32_t hi = p.E - 1;  // last expert whose first tile is not after t
    while (lo < hi) {
      const int32_t mid = (lo + hi + 1) >> 1;
      if (ctl->first[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    x.e = lo;
    t -= ctl->first[lo];
    rows0 = ctl->cut[lo];
    rows1 = ctl->cut[lo + 1];
    if (PROD != kGradW) n_mt = (rows1 - rows0 + kBM - 1) / kBM;
  }
  constexpr int32_t kBand = 16;
  const int32_t band = t / (kBand * p.n_nt), rem = t - band * kBand * p.n_nt;
  const int32_t high = min(kBand, n_mt - band * kBand);
  const int32_t nt = rem / high, mt = band * kBand + rem % high;
  x.n0 = nt * kBN;
  if (PROD == kGradW) {
    x.m0 = mt * kBM;
    x.m_end = p.M;
    x.k0 = rows0;
    x.k_end = rows1;
  } else {
    x.m0 = rows0 + mt * kBM;
    x.m_end = rows1;
    x.k0 = 0;
    x.k_end = p.K;
  }
  x.nk = (x.k_end - x.k0 + kBK - 1) / kBK;
  return x;
}

// The experts' row ranges and tile counts, by warp 0.
template <int PROD>
__device__ __forceinline__ void plan_tiles(const LinearP& p, Ctl* ctl, int lane) {
  if (!p.offsets) {
    if (lane == 0) ctl->first[1] = p.n_mt * p.n_nt;
    return;
  }
  int32_t row = 0, tiles = 0;
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
    int32_t start = __shfl_up_sync(0xFFFFFFFFu, end, 1);
    if (lane == 0) start = row;
    int32_t n = e >= p.E ? 0 : PROD == kGradW ? p.n_mt * p.n_nt : (end - start + kBM - 1) / kBM * p.n_nt;
    const int32_t own = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t u = __shfl_up_sync(0xFFFFFFFFu, n, o);
      if (lane >= o) n += u;
    }
    if (e < p.E) {
      ctl->cut[e] = start;
      ctl->first[e] = tiles + n - own;
    }
    row = __shfl_sync(0xFFFFFFFFu, end, 31);
    tiles += __shfl_sync(0xFFFFFFFFu, n, 31);
  }
  if (lane == 0) {
    ctl->cut[p.E] = row;
    ctl->first[p.E] = tiles;
  }
}

template <int PROD>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ LinearP p) {
  constexpr bool kAmn = PROD == kGradW, kBmn = PROD != kForward;
  constexpr uint32_t kIdesc = kIdescK | (kAmn ? 1u << 15 : 0u) | (kBmn ? 1u << 16 : 0u);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  Ctl* ctl = reinterpret_cast<Ctl*>(stages + kStages * kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 32) {
    prefetch_tensormap(&p.ta);
    prefetch_tensormap(&p.tb);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl->tfull[b], 1);
      mbar_init(&ctl->tempty[b], kEpiWarps);
    }
    mbar_init(&ctl->done, 1);
    fence_barrier_init();
  }
  if (warp == 0) plan_tiles<PROD>(p, ctl, lane);
  if (warp == 1) {
    __syncwarp();
    tc::tmem_alloc(&ctl->tmem, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = ctl->tmem;
  const int32_t tiles = ctl->first[p.offsets ? p.E : 1];

  if (warp == 0) {
    // ---------------------------------------------------------- producer --
    if (lane == 0) {
      int64_t it = 0;
      bool ok = true;
      for (int32_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const Tile x = tile_at<PROD>(p, ctl, t);
        for (int32_t kb = 0; kb < x.nk; ++kb, ++it) {
          const int s = int(it % kStages);
          if (!mbar_wait(&ctl->empty[s], (uint32_t(it / kStages) & 1u) ^ 1u)) {
            atomicOr(&g_err_linear, kErrWaitEmpty);
            ok = false;
            break;
          }
          uint8_t* a = stages + s * kStageBytes;
          uint8_t* b = a + kABytes;
          uint64_t* bar = &ctl->full[s];
          mbar_arrive_expect_tx(bar, kStageBytes);
          const int32_t k = x.k0 + kb * kBK;
          if (kAmn) {
            for (int i = 0; i < kBM / 64; ++i) tma_load_2d(a + i * kBox, &p.ta, x.m0 + 64 * i, k, bar);
          } else {
            tma_load_2d(a, &p.ta, k, x.m0, bar);
          }
          if (PROD == kForward) {
            tma_load_3d(b, &p.tb, k, x.n0, x.e, bar);
          } else if (PROD == kGradX) {
            for (int i = 0; i < kBN / 64; ++i) tma_load_3d(b + i * kBox, &p.tb, x.n0 + 64 * i, k, x.e, bar);
          } else {
            for (int i = 0; i < kBN / 64; ++i) tma_load_2d(b + i * kBox, &p.tb, x.n0 + 64 * i, k, bar);
          }
        }
      }
      // never leave with loads in flight
      for (int64_t j = it - kStages; j < it; ++j) {
        if (j < 0) continue;
        if (!mbar_wait(&ctl->full[j % kStages], uint32_t(j / kStages) & 1u)) atomicOr(&g_err_linear, kErrDrain);
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------------------------- MMA --
    int64_t it = 0;
    int32_t i = 0;
    bool ok = true;
    for (int32_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const Tile x = tile_at<PROD>(p, ctl, t);
      if (x.nk == 0) continue;  // an expert without rows: the epilogue stores zeros
      const int b = i & 1;
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->tempty[b], ((uint32_t(i) >> 1) & 1u) ^ 1u));
      if (!ok) {
        if (lane == 0) atomicOr(&g_err_linear, kErrWaitEmpty);
        break;
      }
      tc::fence_after();
      const uint32_t d = tmem + uint32_t(b * kBN);
      for (int32_t kb = 0; kb < x.nk; ++kb, ++it) {
        const int s = int(it % kStages);
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->full[s], uint32_t(it / kStages) & 1u));
        if (!ok) {
          if (lane == 0) atomicOr(&g_err_linear, kErrWaitFull);
          break;
        }
        uint8_t* stage = stages + s * kStageBytes;
        if (PROD == kGradW) {
          // rows past this expert's: whole 128-byte rows of every box (the
          // swizzle moves 16-byte pieces inside a row only)
          const int32_t have = x.k_end - x.k0 - kb * kBK;
          if (have < kBK) {
            const uint4 zero = make_uint4(0, 0, 0, 0);
            const int32_t n = (kBK - have) * 8;  // 16-byte pieces per box
            for (int32_t q = lane; q < n * ((kBM + kBN) / 64); q += 32)
              *reinterpret_cast<uint4*>(stage + (q / n) * kBox + have * 128 + (q % n) * 16) = zero;
            fence_proxy_async();
          }
          __syncwarp();
        }
        tc::fence_after();
        if (lane == 0) {
          const uint32_t a_addr = smem_u32(stage), b_addr = a_addr + kABytes;
          const uint64_t ad = kAmn ? tc::sw128_mnmajor_desc(a_addr, kBox) : tc::sw128_kmajor_desc(a_addr);
          const uint64_t bd = kBmn ? tc::sw128_mnmajor_desc(b_addr, kBox) : tc::sw128_kmajor_desc(b_addr);
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            tc::mma_bf16(d, ad + k * (kAmn ? 128 : 2), bd + k * (kBmn ? 128 : 2), kIdesc, uint32_t(kb | k));
          tc::commit(&ctl->empty[s]);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (lane == 0) tc::commit(&ctl->tfull[b]);
      ++i;
    }
    if (lane == 0) {
      tc::commit(&ctl->done);
      if (!mbar_wait(&ctl->done, 0)) atomicOr(&g_err_linear, kErrDrain);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- epilogue --
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    int32_t i = 0;
    for (int32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
      const Tile x = tile_at<PROD>(p, ctl, t);
      const int b = i & 1;
      if (x.nk > 0) {
        const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->tfull[b], (uint32_t(i) >> 1) & 1u));
        if (!ok) {
          if (lane == 0) atomicOr(&g_err_linear, kErrWaitFull);
          break;
        }
        tc::fence_after();
        ++i;
      }
      const int32_t row = x.m0 + quarter * 32 + lane;
      const bool row_ok = row < x.m_end;
      uint16_t* out = p.out + (PROD == kGradW ? x.e * p.stride_out : 0) + int64_t(row) * p.ld_out;
      const uint32_t tbase = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(b * kBN);
#pragma unroll 1
      for (int c = half * (kBN / 2); c < (half + 1) * (kBN / 2); c += 32) {
        uint32_t r[32];
        if (x.nk > 0) {
          tc::ld32(tbase + uint32_t(c), r);
          tc::wait_ld();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0;
        }
        const int32_t n = x.n0 + c;
        if (!row_ok || n >= p.N) continue;
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          const int32_t left = p.N - n - j;
          if (left <= 0) break;
          float v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = __uint_as_float(r[j + q]);
          if (PROD == kForward) {
            if (p.bias) {
              const int64_t at = int64_t(x.e) * p.N + n + j;
#pragma unroll
              for (int q = 0; q < 8; ++q)
                if (q < left)
                  v[q] += p.b32 ? __ldg(static_cast<const float*>(p.bias) + at + q)
                                : bf16_of_bits(__ldg(static_cast<const uint16_t*>(p.bias) + at + q));
            }
            if (p.z) store8(p.z + int64_t(row) * p.ld_z + n + j, left, v);
            if (p.act != GLU_ACT_IDENTITY) {
#pragma unroll
              for (int q = 0; q < 8; ++q) v[q] = act_value(p.act, v[q]);
            }
            if (p.residual) {
              float s[8];
              load8(p.residual + int64_t(row) * p.ld_residual + n + j, left, s);
#pragma unroll
              for (int q = 0; q < 8; ++q) v[q] += s[q];
            }
          }
          store8(out + n + j, left, v);
        }
      }
      if (x.nk > 0) {
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->tempty[b]);
      }
    }
    // rows that no expert has
    if (PROD != kGradW && p.offsets) {
      const float zero[8] = {};
      const int64_t chunks = (p.N + 7) / 8, first = ctl->cut[p.E];
      for (int64_t q = int64_t(blockIdx.x) * kEpiWarps * 32 + threadIdx.x - 64; q < (p.rows - first) * chunks;
           q += int64_t(gridDim.x) * kEpiWarps * 32) {
        const int64_t m = first + q / chunks;
        const int32_t c = int32_t(q % chunks) * 8;
        store8(p.out + m * p.ld_out + c, p.N - c, zero);
        if (PROD == kForward && p.z) store8(p.z + m * p.ld_z + c, p.N - c, zero);
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int PROD>
cudaError_t launch_t(LinearP& p, cudaStream_t s, const DevInfo& d) {
  auto kern = linear_kernel<PROD>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  p.n_mt = (p.M + kBM - 1) / kBM;
  p.n_nt = (p.N + kBN - 1) / kBN;
  // by expert the device counts the tiles: no more than one row tile per
  // expert above the dense count
  const int64_t most = PROD == kGradW ? int64_t(p.n_mt) * p.n_nt * p.E
                                      : (int64_t(p.n_mt) + (p.offsets ? p.E : 0)) * p.n_nt;
  const int grid = int(most < d.sms ? most : d.sms);
  return launch_kernel(kern, grid, kThreads, kSmem, s, p);
}

// ------------------------------------------------------- dz and its sums --

constexpr int kDzRows = 128;  // rows of one expert per block

struct DzP {
  const uint16_t *dy, *z;
  uint16_t* dz;  // NULL: not stored
  float* part;   // [slots, N], or NULL
  float* db;
  const int32_t* offsets;
  int64_t ld_dy, ld_z, ld_dz;
  int32_t rows, N, E, act, slots;
};

__device__ __forceinline__ float act_grad(int act, float z) {
  switch (act) {
    case GLU_ACT_SILU: {
      const float s = __fdividef(1.0f, 1.0f + __expf(-z)), q = __fdividef(1.0f, 1.0f + __expf(z));
      return s * fmaf(z, q, 1.0f);
    }
    case GLU_ACT_GELU_TANH: {
      const float z2 = z * z;
      const float u = 1.5957691216057308f * fmaf(0.044715f * z2, z, z);
      const float du = 1.5957691216057308f * fmaf(0.134145f, z2, 1.0f);
      const float s = __fdividef(1.0f, 1.0f + __expf(-u)), q = __fdividef(1.0f, 1.0f + __expf(u));
      return s * fmaf(z * q, du, 1.0f);
    }
    case GLU_ACT_RELU: return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    case GLU_ACT_GELU_ERF: return fmaf(z * 0.3989422804014327f, __expf(-0.5f * z * z), normcdff(z));
    default: return 1.0f;
  }
}

__device__ __forceinline__ int32_t cut_at(const int32_t* offsets, int32_t e, int32_t rows) {
  return e == 0 ? 0 : max(0, min(offsets[e], rows));
}

// Slots of the sums: expert e has those from floor(cut[e] / kDzRows) + e on,
// enough for its rows in parts of kDzRows.  One block per slot and 512
// columns; a thread has two columns of a part's rows.
__global__ void __launch_bounds__(256) dz_kernel(const DzP p) {
  const int32_t slot = blockIdx.x;
  int32_t e = 0, r0 = 0, r1 = p.rows, part = slot;
  if (p.offsets) {
    int32_t lo = 0, hi = p.E - 1;
    while (lo < hi) {
      const int32_t mid = (lo + hi + 1) >> 1;
      if (cut_at(p.offsets, mid, p.rows) / kDzRows + mid <= slot) lo = mid;
      else hi = mid - 1;
    }
    e = lo;
    r0 = cut_at(p.offsets, e, p.rows);
    r1 = max(r0, cut_at(p.offsets, e + 1, p.rows));
    part = slot - r0 / kDzRows - e;
  }
  const int32_t m0 = r0 + part * kDzRows, m1 = min(r1, m0 + kDzRows);
  if (part < 0 || m0 >= m1) return;
  const int32_t c = blockIdx.y * 512 + 2 * threadIdx.x;
  if (c >= p.N) return;
  const bool two = c + 1 < p.N;
  float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 4
  for (int32_t m = m0; m < m1; ++m) {
    float a, b = 0.0f;
    const uint16_t* q = p.dy + m * p.ld_dy + c;
    if (two) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(q);
      a = __uint_as_float(w << 16);
      b = __uint_as_float(w & 0xFFFF0000u);
    } else {
      a = bf16_of_bits(*q);
    }
    if (p.act != GLU_ACT_IDENTITY) {
      const uint16_t* zq = p.z + m * p.ld_z + c;
      if (two) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(zq);
        a *= act_grad(p.act, __uint_as_float(w << 16));
        b *= act_grad(p.act, __uint_as_float(w & 0xFFFF0000u));
      } else {
        a *= act_grad(p.act, bf16_of_bits(*zq));
      }
    }
    if (p.dz) {
      uint16_t* o = p.dz + m * p.ld_dz + c;
      if (two) *reinterpret_cast<uint32_t*>(o) = bf16x2_of(a, b);
      else *o = bits_of_bf16(a);
    }
    s0 += a;
    s1 += b;
  }
  if (p.part) {
    p.part[int64_t(slot) * p.N + c] = s0;
    if (two) p.part[int64_t(slot) * p.N + c + 1] = s1;
  }
}

// db[e] from the slots of expert e.
__global__ void __launch_bounds__(512) db_kernel(const DzP p) {
  __shared__ float sh[16][33];
  const int32_t e = blockIdx.y, c = blockIdx.x * 32 + threadIdx.x;
  int32_t r0 = 0, r1 = p.rows, first = 0;
  if (p.offsets) {
    r0 = cut_at(p.offsets, e, p.rows);
    r1 = max(r0, cut_at(p.offsets, e + 1, p.rows));
    first = r0 / kDzRows + e;
  }
  const int32_t n = (r1 - r0 + kDzRows - 1) / kDzRows;
  float v = 0.0f;
  if (c < p.N)
    for (int32_t i = threadIdx.y; i < n; i += 16) v += p.part[int64_t(first + i) * p.N + c];
  sh[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0 || c >= p.N) return;
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) v += sh[i][threadIdx.x];
  p.db[int64_t(e) * p.N + c] = v;
}

int64_t padded8(int64_t n) { return (n + 7) / 8 * 8; }
int64_t dz_slots(const glu_block_linear_bwd_args& a) { return (a.M + kDzRows - 1) / kDzRows + (a.E > 0 ? a.E : 0); }
size_t dz_bytes(const glu_block_linear_bwd_args& a) {
  return a.act != GLU_ACT_IDENTITY && (a.dx || a.dw) ? size_t(a.M) * padded8(a.N) * 2 : 0;
}

}  // namespace

size_t linear_fwd_workspace(const glu_block_linear_fwd_args&) { return 0; }
size_t linear_bwd_workspace(const glu_block_linear_bwd_args& a) {
  return dz_bytes(a) + (a.db ? size_t(dz_slots(a)) * a.N * 4 : 0);
}

cudaError_t launch_linear_fwd(const glu_block_linear_fwd_args& a, cudaStream_t s, const DevInfo& d) {
  LinearP p;
  memset(&p, 0, sizeof p);
  const int64_t E = a.E > 0 ? a.E : 1;
  cudaError_t e = make_tile_map(&p.ta, a.x, 2, a.K, a.M, a.ld_x * 2, kBK, kBM, 128);
  if (e == cudaSuccess)
    e = make_stack_map(&p.tb, a.w, a.K, a.N, a.ld_w * 2, E, (a.E > 0 ? a.stride_w : a.N * a.ld_w) * 2, kBN);
  if (e != cudaSuccess) return e;
  p.offsets = a.E > 0 ? a.offsets : nullptr;
  p.E = int32_t(E);
  p.rows = p.M = int32_t(a.M);
  p.N = int32_t(a.N);
  p.K = int32_t(a.K);
  p.out = static_cast<uint16_t*>(a.y);
  p.ld_out = a.ld_y;
  p.z = static_cast<uint16_t*>(a.z);
  p.ld_z = a.ld_z;
  p.residual = static_cast<const uint16_t*>(a.residual);
  p.ld_residual = a.ld_residual;
  p.bias = a.bias;
  p.b32 = a.b_fmt == GLU_FMT_FP32;
  p.act = a.act;
  return launch_t<kForward>(p, s, d);
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
    q.act = a.act;
    q.slots = int32_t(dz_slots(a));
    e = launch_kernel(dz_kernel, dim3(unsigned(q.slots), unsigned((a.N + 511) / 512)), 256, 0, s, q);
    if (e != cudaSuccess) return e;
    if (a.db) {
      e = launch_kernel(db_kernel, dim3(unsigned((a.N + 31) / 32), unsigned(E)), dim3(32, 16), 0, s, q);
      if (e != cudaSuccess) return e;
    }
    if (q.dz) dz = q.dz, ld_dz = q.ld_dz;
  }
  LinearP p;
  memset(&p, 0, sizeof p);
  p.offsets = a.E > 0 ? a.offsets : nullptr;
  p.E = int32_t(E);
  p.rows = int32_t(a.M);
  if (a.dx) {
    e = make_tile_map(&p.ta, dz, 2, a.N, a.M, ld_dz * 2, kBK, kBM, 128);
    if (e == cudaSuccess)
      e = make_stack_map(&p.tb, a.w, a.K, a.N, a.ld_w * 2, E, (a.E > 0 ? a.stride_w : a.N * a.ld_w) * 2, kBK);
    if (e != cudaSuccess) return e;
    p.M = int32_t(a.M);
    p.N = int32_t(a.K);
    p.K = int32_t(a.N);
    p.out = static_cast<uint16_t*>(a.dx);
    p.ld_out = a.ld_dx;
    e = launch_t<kGradX>(p, s, d);
    if (e != cudaSuccess) return e;
  }
  if (a.dw) {
    e = make_tile_map(&p.ta, dz, 2, a.N, a.M, ld_dz * 2, 64, kBK, 128);
    if (e == cudaSuccess) e = make_tile_map(&p.tb, a.x, 2, a.K, a.M, a.ld_x * 2, 64, kBK, 128);
    if (e != cudaSuccess) return e;
    p.M = int32_t(a.N);
    p.N = int32_t(a.K);
    p.K = int32_t(a.M);
    p.out = static_cast<uint16_t*>(a.dw);
    p.ld_out = a.ld_dw;
    p.stride_out = a.stride_dw;
    e = launch_t<kGradW>(p, s, d);
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
