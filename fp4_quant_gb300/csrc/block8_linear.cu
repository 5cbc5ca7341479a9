// Products of 8-bit operands with a scale per block of 128 (glu_block8.h), on the
// tcgen05 tensor cores:
//
//   y  = x W^T    summed over K, blocks of 128 columns of x
//   dx = dy W     summed over N
//   dw = dy^T x   summed over the tokens, blocks of 128 rows
//
//   D[i, j] = sum over blocks b of sa(i, b) sb(j, b) sum over k in b of A[i, k] B[j, k]
//
// Tiles and walk are those of the bf16 layers (block_tiles.cuh): 256 rows of D by
// up to 256 columns for a pair of CTAs.  One block of the sum is one slice of the
// ring (128 codes are the 128 bytes of the swizzle) and one accumulator in tensor
// memory: while the tensor cores sum the next block into the other one, eight warps
// read this one, scale it and add it to what they hold in registers, 128 fp32 per
// thread.  Their share of the register file is raised for that (setmaxnreg), the
// other four warps' lowered.  Two of those fetch the scales, block by block ahead.
//
// What a thread has of the accumulator decides what its scales cost.  With the
// tokens as the rows of D (ROWS: many tokens) it has one row of 128 columns, where
// the token's scale and the weight's are one number per block: 4096 x 8192 x 7168
// takes 174 to 191 us with the clocks that the power limit leaves (2760 to 2520
// TFLOP/s), its dx 168 to 187, 32768 rows of 64 uneven experts x 2048 x 2048 153 to 167.  With few tokens they are the columns, whose number the instruction
// leaves free in steps of 32, and so they are in the columns' place for dw, whose
// rows and columns both have scales of their own.  A thread with one row would need
// all the columns' scales then, 128 KB out of shared memory per block at 128 bytes a
// clock (4096 x 8192 x 7168 took 299 us that way, 215 with the scales left out).
// So it reads the accumulator as fragments, a quarter of the columns of four rows
// (203 us; dw of 4096 x 8192 x 7168 258).
//
// What binds is a block's way between the tensor cores and the registers: a block's
// 512 cycles of products, the hand-over to the epilogue's warps and back between the
// CTAs, eight reads of tensor memory; without the additions 166 us, with the
// products and barriers alone 164.  So the epilogue waits for one barrier per block,
// which counts the products and the scales, a block's first chunk is on its way
// behind the last one's additions, accumulators go back by relaxed arrivals between
// tcgen05 fences (release at cluster scope waits for all that a thread has in
// flight: 499 us at first, 301 without), and the results leave through shared memory
// by bulk copies while the next tile is summed (stored from registers 8 us more; dw
// by expert 319 against 258).
#include <cstring>

#include "block8.h"
#include "block_linear.cuh"
#include "block_tiles.cuh"
#include "tc.cuh"
#include "tma.cuh"

namespace gq {
namespace {

constexpr int kBK8 = 128, kStages8 = 4;
constexpr int kOperand8 = kHalf * kBK8;  // 16 KB
constexpr int kStageBytes8 = 2 * kOperand8;
constexpr int kScaleSlots = 2;  // as many as accumulators, whose barriers count the scales too
constexpr int kLoadWarps = 4, kEpiWarps8 = 8;  // loads, products, two of scales; epilogue
constexpr int kThreads8 = (kLoadWarps + kEpiWarps8) * 32;
// 168 registers per thread at launch: 128 x 56 + 256 x 224 = 384 x 168
constexpr int kFewRegs = 56, kManyRegs = 224;
constexpr uint32_t kTmemCols8 = 2 * kTile;
constexpr uint32_t kIdesc8 = tc::idesc_e4m3_f32(kTile, 0);  // the columns are added per tile

struct Scales {
  float col[kTile];
  float row[kHalf];
};
struct Ctl8 {
  uint64_t full[kStages8];   // CTA 0's: its arrival and the bytes of both CTAs
  uint64_t empty[kStages8];  // each CTA's own: the products on its stage are done
  uint64_t tfull[2];         // each CTA's own: a block's sum is complete, and its scales are there
  uint64_t tempty[2];        // CTA 0's: the warps of both have read it
  uint64_t sempty[kScaleSlots];  // each CTA's own: its warps have used the scales
  uint64_t done;             // each CTA's own: all products are done
  uint32_t tmem;
  alignas(16) Scales scales[kScaleSlots];
  TilePlan plan;
};
// A tile's results on their way out, by rows of the output: 256 tokens of 128
// columns (bf16), or 128 rows of 256 (bf16) or of 128 at a time (fp32).  Rows 16
// bytes further apart than they are long: the eight rows of a fragment then begin
// in different banks.
constexpr int kTokenPitch = kHalf * 2 + 16, kRowPitch = kTile * 2 + 16;
constexpr int kOut8 = kTile * kTokenPitch > kHalf * kRowPitch ? kTile * kTokenPitch : kHalf * kRowPitch;
constexpr int kSmem8 = 1024 + kStages8 * kStageBytes8 + kOut8 + int(sizeof(Ctl8));
static_assert(kSmem8 <= 232448, "shared memory per CTA exceeds 227 KB");

__device__ uint32_t g_err_linear8;

struct Linear8P {
  CUtensorMap ta, tb[3];   // tb[i]: boxes of 128 >> i rows, for tiles with fewer columns; dw: tb[0]
  const int32_t* offsets;  // NULL: dense
  int32_t E;               // experts (dense: 1)
  int32_t rows;            // of x (dw: rows that the offsets may reach, dense: of the column forms)
  int32_t width;           // rows of D: N, K (dx) or N
  int32_t cols;            // columns of D of a dw (K)
  int32_t depth;           // summed over (y: K, dx: N)
  int32_t n_at;            // tiles of 256 rows of D
  int32_t most;            // most tokens of a tile (a multiple of 32, up to 256)
  int32_t splits;          // parts of the sum
  // scales: of A's block b and rows of a CTA (y and dx: sa[e sa_e + row / 128 sa_row + b sa_b]; dw: sa[b width + row]),
  // of B's (sb[b ld_sb + column])
  const float *sa, *sb;
  int64_t sa_e, sa_row, sa_b, ld_sb;
  int64_t ld_out, stride_out;
  void* out;
  int32_t f32;             // dw in fp32
  float* part;             // splits > 1: [splits, rows, ld_part]
  int64_t ld_part;
};

struct Tile8 : Tile {
  int32_t a_end;  // ROWS: rows of D end here (of the width: they go on, and are cut where they are stored)
};
// Tile t; a dw sums over its expert's blocks of the column forms.  ROWS: the
// tokens are the rows of D and the width its columns.
template <int PROD, bool ROWS>
__device__ __forceinline__ Tile8 tile8_at(const Linear8P& p, const TilePlan& plan, int32_t t) {
  Tile8 x;
  const bool parts = PROD == kGradW && p.splits > 1;
  const int32_t whole = parts ? t / p.splits : t, split = t - whole * p.splits;
  static_cast<Tile&>(x) = tile_at<PROD, kBK8>(p, plan, whole);
  if (PROD == kGradW && p.offsets) {
    const int32_t rows = x.k_end - x.k0;
    x.k0 = (x.k0 / kBK8 + x.e) * kBK8;
    x.k_end = x.k0 + (rows + kBK8 - 1) / kBK8 * kBK8;
  }
  if (parts) {  // whole blocks, as equal as they go (at most 2^24 of them, and 16 parts)
    const int32_t blocks = (x.k_end - x.k0) / kBK8, first = x.k0 / kBK8;
    x.split = split;
    x.k0 = (first + blocks * split / p.splits) * kBK8;
    x.k_end = (first + blocks * (split + 1) / p.splits) * kBK8;
  }
  x.a_end = p.width;
  if (ROWS) {
    const int32_t a0 = x.a0;
    x.a0 = x.b0;
    x.a_end = x.b_end;
    x.b0 = a0;
    x.b_end = min(p.width, a0 + kTile);
    x.n = kTile;
  }
  return x;
}

// An 8 x 8 block of 16-bit values (lane l: row l / 4, columns 2 (l % 4) and the next) transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Barrier of the epilogue's warps.
__device__ __forceinline__ void epilogue_barrier() { asm volatile("barrier.sync 1, %0;" ::"n"(kEpiWarps8 * 32) : "memory"); }

// `bytes` of an output row from shared memory (both on 16 bytes): whole 16 bytes by
// the copy engine, as part of this thread's bulk group, the rest (elements of
// `size`) by the thread.
__device__ __forceinline__ void put_row(void* out, const uint8_t* row, int32_t bytes, int size) {
  const uint32_t whole = uint32_t(bytes) & ~15u;
  if (whole) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(out), "r"(smem_u32(row)), "r"(whole) : "memory");
  }
  for (int32_t i = int32_t(whole); i < bytes; i += size) {
    if (size == 4) *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(out) + i) = *reinterpret_cast<const uint32_t*>(row + i);
    else *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(out) + i) = *reinterpret_cast<const uint16_t*>(row + i);
  }
}

template <int REGS>
__device__ __forceinline__ void fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}

template <int PROD, bool ROWS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads8, 1) linear8_kernel(const __grid_constant__ Linear8P p) {
  constexpr bool kAmn = !ROWS && PROD != kForward, kBmn = ROWS ? PROD == kGradX : PROD == kGradW;
  constexpr uint32_t kIdesc = kIdesc8 | (kAmn ? 1u << 15 : 0u) | (kBmn ? 1u << 16 : 0u);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* out_rows = stages + kStages8 * kStageBytes8;
  Ctl8* ctl = reinterpret_cast<Ctl8*>(out_rows + kOut8);
  const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int32_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  after_previous();
  if (threadIdx.x == 32) {
    prefetch_tensormap(&p.ta);
    for (int s = 0; s < kStages8; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl->tfull[b], 2);
      mbar_init(&ctl->tempty[b], 2 * kEpiWarps8);
    }
    for (int s = 0; s < kScaleSlots; ++s) mbar_init(&ctl->sempty[s], kEpiWarps8);
    mbar_init(&ctl->done, 1);
    fence_barrier_init();
  }
  plan_tiles<PROD>(p, ctl->plan, warp, lane);
  if (warp == 1) {
    __syncwarp();
    tc::pair_alloc(&ctl->tmem, kTmemCols8);
    tc::pair_relinquish();
  }
  tc::fence_before();
  cluster_sync();
  tc::fence_after();
  const uint32_t tmem = ctl->tmem;
  const int32_t tiles = ctl->plan.first[p.offsets ? p.E : 1] * (PROD == kGradW ? p.splits : 1);

  if (warp < kLoadWarps) {
    fewer_regs<kFewRegs>();
    if (warp == 0) {
      // -------------------------------------------------------- producer --
      int s = 0, held = 0;  // held: stages ever filled, up to all
      uint32_t parity = 0;
      const uint32_t full0 = peer_addr(&ctl->full[0], 0);
      bool ok = true;
      for (int32_t t = pair; t < tiles && ok; t += pairs) {
        const Tile8 x = tile8_at<PROD, ROWS>(p, ctl->plan, t);
        const int32_t a0 = x.a0 + int32_t(rank) * kHalf, half = x.n / 2, b0 = x.b0 + int32_t(rank) * half;
        // the smallest box with the half's columns (more than it needs are not
        // multiplied)
        const int box = half > 64 ? 0 : half > 32 ? 1 : 2;
        const uint32_t bytes = uint32_t(kOperand8 + (kHalf >> box) * kBK8);
        const CUtensorMap* tb = &p.tb[PROD == kGradW ? 0 : box];
        for (int32_t k = x.k0; k < x.k_end; k += kBK8) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->empty[s], parity ^ 1u));
          if (!ok) {
            if (lane == 0) atomicOr(&g_err_linear8, kErrWaitEmpty);
            break;
          }
          if (tc::elect_one()) {
            uint8_t* a = stages + s * kStageBytes8;
            uint8_t* b = a + kOperand8;
            const uint32_t bar = full0 + 8u * uint32_t(s);
            if (rank == 0) mbar_arrive_expect_tx(&ctl->full[s], 2 * bytes);
            if (ROWS) {
              pair_load_2d(a, &p.tb[0], k, a0, bar);
              if (PROD == kForward) pair_load_3d(b, &p.ta, k, b0, x.e, bar);
              else pair_load_3d(b, &p.ta, b0, k, x.e, bar);
            } else if (PROD == kForward) pair_load_3d(a, &p.ta, k, a0, x.e, bar);
            else if (PROD == kGradX) pair_load_3d(a, &p.ta, a0, k, x.e, bar);
            else pair_load_2d(a, &p.ta, a0, k, bar);
            if (PROD == kGradW) pair_load_2d(b, tb, b0, k, bar);
            else if (!ROWS) pair_load_2d(b, tb, k, b0, bar);
          }
          held = max(held, s + 1);
          if (++s == kStages8) s = 0, parity ^= 1u;
        }
      }
      // never leave with loads in flight: the products on each stage's last slice
      // (which waited for its loads) are done
      if (s == held) s = 0, parity ^= 1u;
      for (int j = 0; j < held; ++j) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&ctl->empty[s], parity ^ 1u)) && lane == 0) atomicOr(&g_err_linear8, kErrDrain);
        if (++s == held) s = 0, parity ^= 1u;
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------- MMA --
      int s = 0;
      uint32_t parity = 0, i = 0;  // i: blocks summed
      const uint32_t a_addr = smem_u32(stages);
      const uint64_t ad0 = kAmn ? tc::sw128_mnmajor_desc(a_addr, kOperand8) : tc::sw128_kmajor_desc(a_addr);
      const uint64_t bd0 = kBmn ? tc::sw128_mnmajor_desc(a_addr + kOperand8, kOperand8) : tc::sw128_kmajor_desc(a_addr + kOperand8);
      bool ok = true;
      for (int32_t t = pair; t < tiles && ok && rank == 0; t += pairs) {
        const Tile8 x = tile8_at<PROD, ROWS>(p, ctl->plan, t);
        const uint32_t idesc = kIdesc | (uint32_t(x.n >> 3) << 17);
        for (int32_t k = x.k0; k < x.k_end; k += kBK8) {
          const uint32_t b = i & 1u;
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->full[s], parity));
          if (!ok) {
            if (lane == 0) atomicOr(&g_err_linear8, kErrWaitFull);
            break;
          }
          ok = __all_sync(0xFFFFFFFFu, mbar_wait_relaxed(&ctl->tempty[b], ((i >> 1) & 1u) ^ 1u));
          if (!ok) {
            if (lane == 0) atomicOr(&g_err_linear8, kErrWaitEmpty);
            break;
          }
          tc::fence_after();
          if (tc::elect_one()) {
            const uint64_t ad = ad0 + uint32_t(s * (kStageBytes8 >> 4)), bd = bd0 + uint32_t(s * (kStageBytes8 >> 4));
#pragma unroll
            for (int j = 0; j < kBK8 / 32; ++j)
              tc::pair_mma_e4m3(tmem + b * kTile, ad + j * (kAmn ? 256 : 2), bd + j * (kBmn ? 256 : 2), idesc, uint32_t(j));
            tc::pair_commit(&ctl->empty[s]);
            tc::pair_commit(&ctl->tfull[b]);
          }
          __syncwarp();
          ++i;
          if (++s == kStages8) s = 0, parity ^= 1u;
        }
      }
      __syncwarp();
      if (tc::elect_one()) {  // the lane that issued the products
        if (rank == 0) tc::pair_commit(&ctl->done);
        if (!mbar_wait(&ctl->done, 0)) atomicOr(&g_err_linear8, kErrDrain);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- scales --
      // warp 2 has the even blocks, warp 3 the odd ones; the next one's loads are
      // in flight while one is stored
      uint32_t i = 0;
      bool ok = true;
      for (int32_t t = pair; t < tiles && ok; t += pairs) {
        const Tile8 x = tile8_at<PROD, ROWS>(p, ctl->plan, t);
        const int32_t b0 = x.k0 / kBK8, b1 = (x.k_end + kBK8 - 1) / kBK8;
        const int32_t row0 = x.a0 + int32_t(rank) * kHalf;
        // ROWS: the tokens' are the rows', the weight's one for either half of the columns
        const float* sa = p.sa + (PROD == kGradW ? int64_t(row0) : x.e * p.sa_e + (ROWS ? x.b0 : row0) / kBlock8 * p.sa_row);
        const float* sb = p.sb + (ROWS ? row0 : x.b0);
        float col[8], row[4], next_col[8], next_row[4];
        auto load = [&](int32_t b, float (&c)[8], float (&r)[4]) {
          if (ROWS) {
            c[0] = lane < 2 && x.b0 + kHalf * lane < p.width ? __ldg(sa + b * p.sa_b + lane * p.sa_row) : 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = row0 + 32 * j + lane < x.a_end ? __ldg(sb + int64_t(b) * p.ld_sb + 32 * j + lane) : 0.0f;
            return;
          }
          if (PROD == kGradW) {
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = row0 + 32 * j + lane < p.width ? __ldg(sa + int64_t(b) * p.width + 32 * j + lane) : 0.0f;
          } else {
            r[0] = row0 < p.width ? __ldg(sa + b * p.sa_b) : 0.0f;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) c[j] = x.b0 + 32 * j + lane < x.b_end ? __ldg(sb + int64_t(b) * p.ld_sb + 32 * j + lane) : 0.0f;
        };
        int32_t b = b0 + int32_t((uint32_t(warp - 2) ^ i) & 1u);
        if (b < b1) load(b, col, row);
        for (; b < b1; b += 2) {
          const uint32_t at = i + uint32_t(b - b0);
          const int slot = int(at % kScaleSlots);
          if (b + 2 < b1) load(b + 2, next_col, next_row);
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->sempty[slot], ((at / kScaleSlots) & 1u) ^ 1u));
          if (!ok) {
            if (lane == 0) atomicOr(&g_err_linear8, kErrWaitEmpty);
            break;
          }
          Scales& o = ctl->scales[slot];
          if (ROWS) {
            if (lane < 2) o.col[lane] = col[0];
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) o.col[32 * j + lane] = PROD == kGradW ? col[j] : col[j] * row[0];
          }
          if (ROWS || PROD == kGradW) {
#pragma unroll
            for (int j = 0; j < 4; ++j) o.row[32 * j + lane] = row[j];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->tfull[slot]);
#pragma unroll
          for (int j = 0; j < 8; ++j) col[j] = next_col[j];
#pragma unroll
          for (int j = 0; j < 4; ++j) row[j] = next_row[j];
        }
        i += uint32_t(b1 - b0);
      }
    }
  } else {
    // ---------------------------------------------------------- epilogue --
    more_regs<kManyRegs>();
    const int quarter = warp & 3, group = (warp - kLoadWarps) >> 2;
    const uint32_t tempty0 = peer_addr(&ctl->tempty[0], 0);
    const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16);
    uint32_t i = 0;
    // a warp whose wait gave up waits for nothing more and stores nothing, but keeps
    // to the barriers that it shares with the others
    bool ok = true;
    for (int32_t t = pair; t < tiles; t += pairs) {
      const Tile8 x = tile8_at<PROD, ROWS>(p, ctl->plan, t);
      // acc[q][i][k]: row lane / 4 + 8 i of the warp's 32, columns 8 k + 2 (lane % 4)
      // and the next of the 32 from c0 + 32 q on; ROWS: row `lane`, columns 8 i + 2 k
      // and the next
      float2 acc[4][4][4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[q][j / 4][j % 4] = make_float2(0.0f, 0.0f);
      const int c0 = group * (x.n / 2), c1 = c0 + x.n / 2;  // this group's columns
      const int chunks = x.n > kTile / 2 ? 4 : 2;  // of 32 columns; what is read past c1 is not stored
      uint32_t r[2][2][16];
      float2 s[2][4];
      // block i's sum and scales are there
      auto ready = [&] {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->tfull[i & 1u], (i >> 1) & 1u));
        if (!ok && lane == 0) atomicOr(&g_err_linear8, kErrWaitFull);
        tc::fence_after();
      };
      auto fetch = [&](int q) {
        const uint32_t at = lanes + (i & 1u) * kTile + uint32_t(c0 + 32 * q);
        if (ROWS) {
          tc::ld32(at, reinterpret_cast<uint32_t(&)[32]>(r[q & 1]));
          return;
        }
        tc::ld16x32(at, r[q & 1][0]);
        tc::ld16x32(at + (16u << 16), r[q & 1][1]);
        const float* col = ctl->scales[i % kScaleSlots].col + c0 + 32 * q + 2 * (lane & 3);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[q & 1][j] = *reinterpret_cast<const float2*>(col + 8 * j);
      };
      if (x.k0 < x.k_end && ok) {
        ready();
        if (ok) fetch(0);
      }
      for (int32_t k = x.k0; k < x.k_end && ok; k += kBK8) {
        const int slot = int(i % kScaleSlots);
        const Scales& sc = ctl->scales[slot];
        float row[4];
        if (ROWS) row[0] = sc.row[quarter * 32 + lane] * sc.col[group];
        if (PROD == kGradW) {
#pragma unroll
          for (int j = 0; j < 4; ++j) row[j] = sc.row[quarter * 32 + (lane >> 2) + 8 * j];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (q >= chunks) break;
          tc::wait_ld(r[q & 1]);
          // the next chunk, of the next block behind the last one, is on its way
          // while this one is added
          if (q + 1 < chunks) {
            fetch(q + 1);
          } else {
            tc::fence_before();
            __syncwarp();
            if (lane == 0) peer_arrive_relaxed(tempty0 + 8u * (i & 1u));
            ++i;
            if (k + kBK8 < x.k_end) {
              ready();
              if (ok) fetch(0);
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint32_t* v = ROWS ? &r[q & 1][y >> 1][8 * (y & 1) + 2 * j] : &r[q & 1][y >> 1][4 * j + 2 * (y & 1)];
              float2 d = make_float2(__uint_as_float(v[0]), __uint_as_float(v[1]));
              if (ROWS) {
                acc[q][y][j] = fma_2(d, both(row[0]), acc[q][y][j]);
                continue;
              }
              if (PROD == kGradW) d = mul_2(d, both(row[y]));
              acc[q][y][j] = fma_2(d, s[q & 1][j], acc[q][y][j]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->sempty[slot]);
      }
      const int32_t row0 = x.a0 + int32_t(rank) * kHalf + quarter * 32;  // of D: this warp's 32
      const int32_t b_end = min(x.b_end, x.b0 + c1);                     // of this group
      if (!ROWS && PROD != kGradW && p.splits > 1) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int32_t n = row0 + (lane >> 2) + 8 * y, token = x.b0 + c0 + 32 * q + 8 * j + 2 * (lane & 3);
              float* out = p.part + (int64_t(x.split) * p.rows + token) * p.ld_part + n;
              if (!ok) continue;
              if (n < p.width && token < b_end) out[0] = acc[q][y][j].x;
              if (n < p.width && token + 1 < b_end) out[p.ld_part] = acc[q][y][j].y;
            }
        continue;
      }
      // into shared memory, where the last tile's rows have left, and out from there
      // while the next tile is summed
      const int er = (warp - kLoadWarps) * 32 + lane;  // 0 .. 255
      const int32_t cta0 = x.a0 + int32_t(rank) * kHalf;  // of D: this CTA's rows
      if (ROWS) {
        bulk_wait_read0();
        epilogue_barrier();
        uint8_t* row = out_rows + (quarter * 32 + lane) * kRowPitch + c0 * 2;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float2(&v)[4] = acc[q][y];
            *reinterpret_cast<uint4*>(row + (32 * q + 8 * y) * 2) =
                make_uint4(bf16x2_of(v[0].x, v[0].y), bf16x2_of(v[1].x, v[1].y), bf16x2_of(v[2].x, v[2].y), bf16x2_of(v[3].x, v[3].y));
          }
        fence_proxy_async();
        epilogue_barrier();
        if (ok && er < kHalf && cta0 + er < x.a_end)
          put_row(static_cast<uint16_t*>(p.out) + int64_t(cta0 + er) * p.ld_out + x.b0, out_rows + er * kRowPitch, (x.b_end - x.b0) * 2, 2);
        bulk_commit();
      } else if (PROD != kGradW) {
        bulk_wait_read0();
        epilogue_barrier();
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (c0 + 32 * q + 8 * j < c1) {
#pragma unroll
              for (int y = 0; y < 4; ++y)  // an 8 x 8 block: rows of D by tokens, transposed
                *reinterpret_cast<uint32_t*>(out_rows + (c0 + 32 * q + 8 * j + (lane >> 2)) * kTokenPitch +
                                             (quarter * 32 + 8 * y + 2 * (lane & 3)) * 2) =
                    transpose8x8(bf16x2_of(acc[q][y][j].x, acc[q][y][j].y));
          }
        fence_proxy_async();
        epilogue_barrier();
        const int32_t left = min(p.width - cta0, int32_t(kHalf));
        if (ok && x.b0 + er < x.b_end && left > 0)
          put_row(static_cast<uint16_t*>(p.out) + int64_t(x.b0 + er) * p.ld_out + cta0, out_rows + er * kTokenPitch, left * 2, 2);
        bulk_commit();
      } else {
        // the parts of a split sum follow each other
        const int64_t base = (int64_t(x.split) * p.E + x.e) * p.stride_out + int64_t(cta0) * p.ld_out + x.b0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // fp32: the columns of either group in turn
          if (!p.f32 && h == 1) break;
          bulk_wait_read0();
          epilogue_barrier();
          if (!p.f32 || group == h) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                uint8_t* row = out_rows + (quarter * 32 + (lane >> 2) + 8 * y) * kRowPitch;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int c = 32 * q + 8 * j + 2 * (lane & 3);
                  if (p.f32) *reinterpret_cast<float2*>(row + c * 4) = acc[q][y][j];
                  else *reinterpret_cast<uint32_t*>(row + (c0 + c) * 2) = bf16x2_of(acc[q][y][j].x, acc[q][y][j].y);
                }
              }
          }
          fence_proxy_async();
          epilogue_barrier();
          const int32_t first = p.f32 ? kHalf * h : 0, left = min(x.b_end - x.b0 - first, p.f32 ? kHalf : kTile);
          if (ok && er < kHalf && cta0 + er < p.width && left > 0) {
            const int64_t at = base + er * p.ld_out + first;
            if (p.f32) put_row(static_cast<float*>(p.out) + at, out_rows + er * kRowPitch, left * 4, 4);
            else put_row(static_cast<uint16_t*>(p.out) + at, out_rows + er * kRowPitch, left * 2, 2);
          }
          bulk_commit();
        }
      }
    }
    bulk_wait0();
    // rows that no expert has
    if (PROD != kGradW && p.offsets) {
      const float zero[8] = {};
      const int64_t chunks = (p.width + 7) / 8, first = ctl->plan.cut[p.E];
      for (int64_t q = int64_t(blockIdx.x) * kEpiWarps8 * 32 + threadIdx.x - kLoadWarps * 32; q < (p.rows - first) * chunks;
           q += int64_t(gridDim.x) * kEpiWarps8 * 32) {
        const int64_t m = first + q / chunks;
        const int32_t c = int32_t(q % chunks) * 8;
        store8(static_cast<uint16_t*>(p.out) + m * p.ld_out + c, p.width - c, zero);
      }
    }
  }
  __syncwarp();
  tc::fence_before();
  cluster_sync();
  if (warp == 1) {
    tc::fence_after();
    tc::pair_dealloc(tmem, kTmemCols8);
  }
}

std::atomic<int> known8[64];  // pairs at once, alike for every product

template <int PROD, bool ROWS>
cudaError_t launch8(Linear8P& p, cudaStream_t s, const DevInfo& d) {
  auto kern = linear8_kernel<PROD, ROWS>;
  static SmemLimit limit;
  cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern), kSmem8);
  if (e != cudaSuccess) return e;
  p.n_at = (p.width + kTile - 1) / kTile;
  // by expert the device counts the tiles: no more than one token tile per
  // expert above the dense count
  const int64_t most = PROD == kGradW ? int64_t(p.n_at) * ((p.cols + kTile - 1) / kTile) * p.E * p.splits
                                      : p.n_at * ((int64_t(p.rows) + p.most - 1) / p.most + (p.offsets ? p.E : 0)) * p.splits;
  int pairs = 0;
  e = pairs_at_once(known8, reinterpret_cast<const void*>(kern), kThreads8, kSmem8, d, &pairs);
  if (e != cudaSuccess) return e;
  if (most < pairs) pairs = int(most);
  return launch_kernel(kern, 2 * pairs, kThreads8, kSmem8, s, p, true);
}

// How the tokens of y or dx are cut into tiles: `rows`, as the rows of D, 256 at a
// time, or as its columns, at most `most` at a time and the sum in parts; a function
// of the shape alone (76 pairs).  As rows a thread has one token, whose scale and the
// weight's are one number per block.  By expert from 128 tokens per W on: with 64
// experts x 2048 x 2048 64 rows each take 78 us as rows and 76 as columns, 128 rows 80
// and 80, 256 rows 109 and 117, 512 158 and 180.  Dense the plan with the least
// estimated time: a block of the sum takes 0.42 us with the tokens as rows (7168 deep,
// 4096 x 8192: 174 us), as columns 0.4 us for 32 of them and 0.55 for 256 (8192 deep,
// 7168 wide: one part for 32 tokens 31 us, two parts, as the plan has it, 22.5; 4096
// tokens 203), the busiest pair's tiles follow each other, and the join of split sums
// reads and writes the fp32 parts.
struct TokenPlan8 {
  int most, splits;
  bool rows;
};
TokenPlan8 token_plan8(int64_t rows, int64_t width, int64_t depth) {
  const int64_t at = (width + kTile - 1) / kTile, blocks = blocks8(depth);
  TokenPlan8 best = {kTile, 1, rows >= 128};
  double least = best.rows ? double((at * ((rows + kTile - 1) / kTile) + 75) / 76) * (double(blocks) * 0.42 + 1.5) : 1e30;
  for (int n = 1; n <= 8 && blocks / n >= 4; ++n)
    for (int most = kTile; most >= 64; most -= kStep) {
      const int64_t bt = (rows + most - 1) / most, each = ((rows + bt - 1) / bt + kStep - 1) / kStep * kStep;
      double us = double((at * bt * n + 75) / 76) * (double((blocks + n - 1) / n) * (0.38 + 0.17 * double(each) / kTile) + 1.5);
      if (n > 1) us += 3.0 + double(n) * double(rows) * double(width) * 8e-6 / 4.0;
      if (us < least * 0.98) least = us, best = {most, n, false};
    }
  return best;
}
TokenPlan8 plan8(const glu_block8_linear_args& a) {
  if (a.E > 0 || linear8_few(a)) return {kTile, 1, a.M >= 128 * int64_t(a.E)};
  return a.grad ? token_plan8(a.M, a.K, a.N) : token_plan8(a.M, a.N, a.K);
}

// dw from the fp32 parts of split sums, added in order: a thread has eight columns of
// a row.
struct JoinDwP {
  const float* part;  // [splits, E N, ld_part]
  void* dw;
  int64_t ld_part, ld_dw, stride_dw, rows;
  int32_t N, K, splits, f32;
};
__global__ void __launch_bounds__(256) join_dw8_kernel(const __grid_constant__ JoinDwP p) {
  const int64_t chunks = (p.K + 7) / 8, q = int64_t(blockIdx.x) * 256 + threadIdx.x;
  after_previous();
  if (q >= p.rows * chunks) return;
  const int64_t row = q / chunks, e = row / p.N;
  const int32_t c = int32_t(q - row * chunks) * 8;
  float v[8] = {};
  for (int i = 0; i < p.splits; ++i) {  // the parts' rows are whole chunks; what lies past K in them is not stored
    const float4* f = reinterpret_cast<const float4*>(p.part + (i * p.rows + row) * p.ld_part + c);
    const float4 a = f[0], b = f[1];
    v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w, v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
  }
  const int64_t at = e * p.stride_dw + (row - e * p.N) * p.ld_dw + c;
  const int32_t left = p.K - c;
  if (!p.f32) {
    store8(static_cast<uint16_t*>(p.dw) + at, left, v);
  } else {
    float* o = static_cast<float*>(p.dw) + at;  // rows begin on 16 bytes
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) o[i] = v[i];
  }
}
int64_t part_ld8(int64_t K) { return (K + 7) / 8 * 8; }

// Parts of a dw's token sum, where its tiles are fewer than the 76 pairs: the number
// with the least estimated time.  A block of the sum takes 0.67 us, a tile's results 2,
// the join reads and writes the parts (64 MB at most).
int dw_splits8(const glu_block8_linear_dw_args& a) {
  const int64_t E = a.E > 0 ? a.E : 1, tiles = (a.N + kTile - 1) / kTile * ((a.K + kTile - 1) / kTile) * E;
  const int64_t blocks = (a.C - (a.E > 0 ? E : 0)) / E + 1, size = E * a.N * part_ld8(a.K) * 4;
  int best = 1;
  double least = 1e30;
  for (int n = 1; n <= 16 && (n == 1 || (blocks / n >= 2 && n * size <= (int64_t(64) << 20))); ++n) {
    double us = double((tiles * n + 75) / 76) * (double((blocks + n - 1) / n) * 0.67 + 2.0);
    if (n > 1) us += 3.0 + double(n) * double(size) * 2e-6 / 4.0;
    if (us < least * 0.95) least = us, best = n;
  }
  return best;
}

}  // namespace

size_t linear8_dw_workspace(const glu_block8_linear_dw_args& a) {
  const int n = dw_splits8(a);
  return n > 1 ? size_t(n) * size_t(a.E > 0 ? a.E : 1) * size_t(a.N) * size_t(part_ld8(a.K)) * 4 : 0;
}

size_t linear8_workspace(const glu_block8_linear_args& a) {
  const int splits = plan8(a).splits;
  return splits > 1 ? size_t(splits) * size_t(a.M) * size_t(((a.grad ? a.K : a.N) + 7) / 8 * 8) * 4 : 0;
}

cudaError_t launch_linear8(const glu_block8_linear_args& a, cudaStream_t s, const DevInfo& d) {
  if (linear8_few(a)) return launch_linear8_few(a, s);
  Linear8P p;
  memset(&p, 0, sizeof p);
  const TokenPlan8 plan = plan8(a);
  const bool grad = a.grad != 0;
  const int64_t E = a.E > 0 ? a.E : 1, depth = grad ? a.N : a.K;
  cudaError_t e = make_byte_stack_map(&p.ta, a.wq, a.K, a.N, a.ld_w, E, a.E > 0 ? a.stride_w : a.N * a.ld_w, kHalf);
  for (int i = 0; i < 3 && e == cudaSuccess; ++i) e = make_tile_map(&p.tb[i], a.xq, 1, depth, a.M, a.ld_x, kBK8, kHalf >> i, 128);
  if (e != cudaSuccess) return e;
  p.offsets = a.E > 0 ? a.offsets : nullptr;
  p.E = int32_t(E);
  p.rows = int32_t(a.M);
  p.width = int32_t(grad ? a.K : a.N);
  p.depth = int32_t(depth);
  p.most = plan.most;
  p.splits = plan.splits;
  p.part = static_cast<float*>(a.workspace);
  p.ld_part = (p.width + 7) / 8 * 8;
  p.sa = a.ws;
  p.sa_e = blocks8(a.N) * blocks8(a.K);
  p.sa_row = grad ? 1 : blocks8(a.K);
  p.sa_b = grad ? blocks8(a.K) : 1;
  p.sb = a.xs;
  p.ld_sb = a.M;
  p.out = a.y;
  p.ld_out = a.ld_y;
  if (plan.rows) return grad ? launch8<kGradX, true>(p, s, d) : launch8<kForward, true>(p, s, d);
  e = grad ? launch8<kGradX, false>(p, s, d) : launch8<kForward, false>(p, s, d);
  if (e != cudaSuccess || p.splits == 1) return e;
  glu_block_linear_fwd_args j = {};  // the join of a bf16 layer without bias, activation and residual
  j.act = GLU_ACT_IDENTITY;
  j.b_fmt = GLU_FMT_BF16;
  j.M = a.M;
  j.N = p.width;
  j.ld_y = a.ld_y;
  j.y = a.y;
  return launch_linear_join(j, p.part, p.splits, s);
}

cudaError_t launch_linear8_dw(const glu_block8_linear_dw_args& a, cudaStream_t s, const DevInfo& d) {
  Linear8P p;
  memset(&p, 0, sizeof p);
  const int64_t rows = a.C * kBlock8;
  cudaError_t e = make_tile_map(&p.ta, a.dyq, 1, a.N, rows, a.ld_dy, 128, kBK8, 128);
  if (e == cudaSuccess) e = make_tile_map(&p.tb[0], a.xq, 1, a.K, rows, a.ld_x, 128, kBK8, 128);
  if (e != cudaSuccess) return e;
  p.offsets = a.E > 0 ? a.offsets : nullptr;
  p.E = int32_t(a.E > 0 ? a.E : 1);
  // M / 128 + E blocks: the last row of M at most, so that no expert's blocks pass C
  p.rows = int32_t(a.E > 0 ? (a.C - a.E) * kBlock8 + kBlock8 - 1 : rows);
  p.width = int32_t(a.N);
  p.cols = int32_t(a.K);
  p.most = kTile;
  p.splits = dw_splits8(a);
  p.sa = a.dys;
  p.sb = a.xs;
  p.ld_sb = a.K;
  p.out = a.dw;
  p.ld_out = a.ld_dw;
  p.stride_out = a.E > 0 ? a.stride_dw : 0;
  p.f32 = a.dw_fmt == GLU_FMT_FP32;
  if (p.splits == 1) return launch8<kGradW, false>(p, s, d);
  JoinDwP j;
  j.part = static_cast<const float*>(a.workspace);
  j.dw = a.dw;
  j.ld_part = part_ld8(a.K);
  j.ld_dw = a.ld_dw;
  j.stride_dw = p.stride_out;
  j.rows = int64_t(p.E) * a.N;
  j.N = p.width;
  j.K = p.cols;
  j.splits = p.splits;
  j.f32 = p.f32;
  p.out = a.workspace;
  p.ld_out = j.ld_part;
  p.stride_out = a.N * j.ld_part;
  p.f32 = 1;
  e = launch8<kGradW, false>(p, s, d);
  if (e != cudaSuccess) return e;
  return launch_kernel(join_dw8_kernel, unsigned((j.rows * ((a.K + 7) / 8) + 255) / 256), 256, 0, s, j, true);
}

cudaError_t read_err_linear8(uint32_t* v, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(v, g_err_linear8, sizeof(uint32_t));
  if (e == cudaSuccess && clear) {
    const uint32_t z = 0;
    e = cudaMemcpyToSymbol(g_err_linear8, &z, sizeof(uint32_t));
  }
  return e;
}

}  // namespace gq
