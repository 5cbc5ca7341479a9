// What stands around the products of the linear layers (glu_block.h): y of few
// tokens, the join of split sums, and dz with its sums over rows.
#include <type_traits>

#include "block_act.cuh"
#include "block_linear.cuh"
#include "block_util.cuh"

namespace gq {
namespace {

// ------------------------------------------------------------ few tokens --
//
// y = act(x W^T + b) + residual for up to 16 tokens: bound by reading W once (2
// N K bytes).  A block has 16 rows of W; its warps share the sum over K, each
// with a part of its own, and join in a fixed order.  The products are mma.sync
// (16 rows x 8 tokens x 16): their rate does not matter here, and their operand
// layout is met without moving data between lanes.  A lane holds eight
// consecutive k of rows g and g + 8 (g = lane / 4), from k0 + 8 (lane % 4) on;
// the sum's order is free, so words 0, 1 of it serve as the instruction's k =
// 2 t .. and 2 t + 8 .. for one instruction, words 2, 3 for the next, with x
// taken the same way.  Every lane copies what it will use itself, 16 bytes at a
// time, into slots of shared memory that only it reads (cp.async), so a warp
// keeps several steps of 32 k in flight without registers or barriers.
constexpr int kFewWarps = 8;

struct FewP {
  const uint16_t *x, *w, *residual;
  const void* bias;
  uint16_t *y, *z;
  int64_t ld_x, ld_w, ld_residual, ld_y, ld_z;
  int32_t M, N, K, b32;
};

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first n (as far as 1..8) elements from k of a row to a slot, the rest 0.
__device__ __forceinline__ void few_copy(uint4* slot, const uint16_t* row, int32_t k, int32_t n) {
  const uint32_t bytes = n >= 8 ? 16u : n > 0 ? 2u * uint32_t(n) : 0u;
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(uint32_t(__cvta_generic_to_shared(slot))),
               "l"(bytes ? row + k : row), "r"(bytes)
               : "memory");
}

// TT: groups of eight tokens; DEEP: slots, one more than the steps in flight.
template <int TT, int DEEP>
constexpr int few_smem() {
  const int ring = kFewWarps * DEEP * (2 + TT) * 32 * 16, sums = kFewWarps * 16 * (8 * TT + 1) * 4;
  return ring > sums ? ring : sums;
}

template <int ACT, int TT, int DEEP>
__global__ void __launch_bounds__(kFewWarps * 32) few_kernel(const FewP p) {
  extern __shared__ __align__(16) uint4 ring[];  // [warps][DEEP][2 + TT][32], then the sums
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t8 = 8 * (lane & 3);
  const int32_t n0 = blockIdx.x * 16;
  // rows past N are read as the last one and not stored
  const uint16_t* w0 = p.w + int64_t(min(n0 + g, p.N - 1)) * p.ld_w;
  const uint16_t* w1 = p.w + int64_t(min(n0 + g + 8, p.N - 1)) * p.ld_w;
  float c[TT][4] = {};
  after_previous();
  // this warp's part of K, in steps of 32
  const int32_t steps = (p.K + 31) / 32, s0 = steps * warp / kFewWarps, s1 = steps * (warp + 1) / kFewWarps;
  uint4* mine = ring + warp * DEEP * (2 + TT) * 32 + lane;
  auto copy = [&](int32_t s, int slot) {
    if (s < s1) {
      const int32_t k = s * 32 + t8, left = p.K - k;
      uint4* q = mine + slot * (2 + TT) * 32;
      few_copy(q, w0, k, left);
      few_copy(q + 32, w1, k, left);
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        const int32_t m = 8 * j + g;
        few_copy(q + (2 + j) * 32, p.x + int64_t(min(m, p.M - 1)) * p.ld_x, k, m < p.M ? left : 0);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < DEEP - 1; ++i) copy(s0 + i, i);
  int slot = 0;
  for (int32_t s = s0; s < s1; ++s) {
    asm volatile("cp.async.wait_group %0;" ::"n"(DEEP - 2) : "memory");
    const uint4* q = mine + slot * (2 + TT) * 32;
    const uint4 a = q[0], b = q[32];
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      const uint4 v = q[(2 + j) * 32];
      mma_16x8x16(c[j], a.x, b.x, a.y, b.y, v.x, v.y);
      mma_16x8x16(c[j], a.z, b.z, a.w, b.w, v.z, v.w);
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
    const int tok = 8 * j + 2 * (lane & 3);
    sums[warp][g][tok] = c[j][0];
    sums[warp][g][tok + 1] = c[j][1];
    sums[warp][g + 8][tok] = c[j][2];
    sums[warp][g + 8][tok + 1] = c[j][3];
  }
  __syncthreads();
  for (int q = threadIdx.x; q < 16 * p.M; q += kFewWarps * 32) {
    const int r = q & 15, m = q >> 4;
    const int32_t n = n0 + r;
    if (n >= p.N) continue;
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kFewWarps; ++i) v += sums[i][r][m];
    if (p.bias) v += p.b32 ? static_cast<const float*>(p.bias)[n] : bf16_of_bits(static_cast<const uint16_t*>(p.bias)[n]);
    if (p.z) p.z[m * p.ld_z + n] = bits_of_bf16(v);
    v = act_value<ACT>(v);
    if (p.residual) v += bf16_of_bits(p.residual[m * p.ld_residual + n]);
    p.y[m * p.ld_y + n] = bits_of_bf16(v);
  }
}

template <int ACT, int TT, int DEEP>
cudaError_t launch_few_d(const FewP& p, cudaStream_t s) {
  constexpr int smem = few_smem<TT, DEEP>();
  auto kern = few_kernel<ACT, TT, DEEP>;
  static SmemLimit limit;
  const cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, unsigned((p.N + 15) / 16), kFewWarps * 32, smem, s, p, true);
}

// Slots by how many blocks share an SM: what is in flight per SM stays about
// the same, and all blocks are there at once up to four per SM.
template <int ACT, int TT>
cudaError_t launch_few_t(const FewP& p, cudaStream_t s) {
  const int blocks = (p.N + 15) / 16;
  if (blocks <= 152) return launch_few_d<ACT, TT, 12 / TT>(p, s);
  if (blocks <= 304) return launch_few_d<ACT, TT, 8 / TT>(p, s);
  return launch_few_d<ACT, TT, 4>(p, s);
}
template <int ACT>
cudaError_t launch_few_a(const FewP& p, cudaStream_t s) {
  return p.M <= 8 ? launch_few_t<ACT, 1>(p, s) : launch_few_t<ACT, 2>(p, s);
}

// ------------------------------------------------- the join of split sums --

struct JoinP {
  const float* part;  // [splits, M, ld]
  const uint16_t* residual;
  const void* bias;
  uint16_t *y, *z;
  int64_t M, N, ld, ld_residual, ld_y, ld_z;
  int32_t splits, b32;
};

// One thread per eight columns of a token, the parts added in order.
template <int ACT>
__global__ void __launch_bounds__(256) linear_join_kernel(const JoinP p) {
  const int64_t chunks = (p.N + 7) / 8, q = int64_t(blockIdx.x) * 256 + threadIdx.x;
  after_previous();
  if (q >= p.M * chunks) return;
  const int64_t m = q / chunks;
  const int32_t c = int32_t(q % chunks) * 8, left = int32_t(p.N) - c;
  F8 v = zeros();
  for (int i = 0; i < p.splits; ++i) {  // the parts' rows are whole chunks; what lies past N in them is not stored
    const float4* f = reinterpret_cast<const float4*>(p.part + (i * p.M + m) * p.ld + c);
    const float4 a = f[0], b = f[1];
    v.v[0] = add_2(v.v[0], make_float2(a.x, a.y));
    v.v[1] = add_2(v.v[1], make_float2(a.z, a.w));
    v.v[2] = add_2(v.v[2], make_float2(b.x, b.y));
    v.v[3] = add_2(v.v[3], make_float2(b.z, b.w));
  }
  if (p.bias) {
    float b[8];
    vec8(p.bias, p.b32, c, left, 0.0f, b);
    const F8 f = pairs(b);
#pragma unroll
    for (int i = 0; i < 4; ++i) v.v[i] = add_2(v.v[i], f.v[i]);
  }
  if (p.z) store8<true>(p.z + m * p.ld_z + c, left, v);
  if (ACT != GLU_ACT_IDENTITY) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v.v[i] = make_float2(act_value<ACT>(v.v[i].x), act_value<ACT>(v.v[i].y));
  }
  if (p.residual) {
    const F8 f = pairs(raw8(p.residual + m * p.ld_residual + c, left));
#pragma unroll
    for (int i = 0; i < 4; ++i) v.v[i] = add_2(v.v[i], f.v[i]);
  }
  store8<true>(p.y + m * p.ld_y + c, left, v);
}

// ------------------------------------------------------- dz and its sums --

__device__ __forceinline__ int32_t cut_at(const int32_t* offsets, int32_t e, int32_t rows) {
  return e == 0 ? 0 : max(0, min(offsets[e], rows));
}

// Slots of the sums: expert e has those from floor(cut[e] / kDzRows) + e on,
// enough for its rows in parts of kDzRows.  One block per slot and 256
// columns: 32 threads of eight columns each by eight rows at a time, four
// rows' loads in flight per thread; the eight sums of a column are joined in
// a fixed order.  Bound by DRAM: dy and z read, dz written, 6 bytes per
// element.
constexpr int kDzCols = 256, kDzDeep = 4;

template <int ACT>
__global__ void __launch_bounds__(256) dz_kernel(const DzP p) {
  __shared__ float sh[8][kDzCols + 8];
  const int32_t slot = blockIdx.x;
  int32_t e = 0, r0 = 0, r1 = p.rows, part = slot;
  after_previous();
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
  const int32_t c = blockIdx.y * kDzCols + 8 * threadIdx.x, left = p.N - c;
  F8 sum = zeros();
  // Whole chunks and the one in which the width ends apart: a choice at each
  // load would hold back the ones after it.
  auto walk = [&](auto whole) {
    for (int32_t m = m0 + threadIdx.y; m < m1; m += 8 * kDzDeep) {
      uint4 a[kDzDeep], z[kDzDeep];
#pragma unroll
      for (int i = 0; i < kDzDeep; ++i) {
        const int64_t row = m + 8 * i;
        if (row >= m1) continue;
        a[i] = raw8(p.dy + row * p.ld_dy + c, decltype(whole)::value ? 8 : left);
        if (ACT != GLU_ACT_IDENTITY) z[i] = raw8(p.z + row * p.ld_z + c, decltype(whole)::value ? 8 : left);
      }
#pragma unroll
      for (int i = 0; i < kDzDeep; ++i) {
        const int64_t row = m + 8 * i;
        if (row >= m1) continue;
        F8 d = pairs(a[i]);
        if (ACT != GLU_ACT_IDENTITY) {
          const uint32_t v[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
#pragma unroll
          for (int q = 0; q < 4; ++q) d.v[q] = mul_2(d.v[q], act_grad_of<ACT>(v[q]));
          // kept in L2: the products read it next
          if (p.dz) *reinterpret_cast<uint4*>(p.dz + row * p.ld_dz + c) = packed(d);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) sum.v[q] = add_2(sum.v[q], d.v[q]);
      }
    }
  };
  if (left >= 8) walk(std::true_type());
  else if (left > 0) walk(std::false_type());
  if (!p.part) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) *reinterpret_cast<float2*>(&sh[threadIdx.y][8 * threadIdx.x + 2 * q]) = sum.v[q];
  __syncthreads();
  const int32_t t = threadIdx.y * 32 + threadIdx.x, col = blockIdx.y * kDzCols + t;
  if (col >= p.N) return;
  float v = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v += sh[i][t];
  p.part[int64_t(slot) * p.N + col] = v;
}

// db[e] from the slots of expert e.
__global__ void __launch_bounds__(512) db_kernel(const DzP p) {
  __shared__ float sh[16][33];
  const int32_t e = blockIdx.y, c = blockIdx.x * 32 + threadIdx.x;
  int32_t r0 = 0, r1 = p.rows, first = 0;
  after_previous();
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

}  // namespace

// Up to 16 tokens: at 7168 x 8192 with W from DRAM this takes 19.9 us for one
// token (5.9 TB/s), 20.3 for eight and 23.2 for 16, where every block's own
// read of x begins to count; the pairs' tiles take 27 us from 1 to 64.
bool linear_few(const glu_block_linear_fwd_args& a) { return a.E == 0 && a.M <= 16; }

cudaError_t launch_linear_few(const glu_block_linear_fwd_args& a, cudaStream_t s) {
  FewP p;
  p.x = static_cast<const uint16_t*>(a.x);
  p.w = static_cast<const uint16_t*>(a.w);
  p.residual = static_cast<const uint16_t*>(a.residual);
  p.bias = a.bias;
  p.y = static_cast<uint16_t*>(a.y);
  p.z = static_cast<uint16_t*>(a.z);
  p.ld_x = a.ld_x;
  p.ld_w = a.ld_w;
  p.ld_residual = a.ld_residual;
  p.ld_y = a.ld_y;
  p.ld_z = a.ld_z;
  p.M = int32_t(a.M);
  p.N = int32_t(a.N);
  p.K = int32_t(a.K);
  p.b32 = a.b_fmt == GLU_FMT_FP32;
  switch (a.act) {
    case GLU_ACT_SILU: return launch_few_a<GLU_ACT_SILU>(p, s);
    case GLU_ACT_GELU_TANH: return launch_few_a<GLU_ACT_GELU_TANH>(p, s);
    case GLU_ACT_RELU: return launch_few_a<GLU_ACT_RELU>(p, s);
    case GLU_ACT_GELU_ERF: return launch_few_a<GLU_ACT_GELU_ERF>(p, s);
    default: return launch_few_a<GLU_ACT_IDENTITY>(p, s);
  }
}

cudaError_t launch_linear_join(const glu_block_linear_fwd_args& a, const float* part, int splits, cudaStream_t s) {
  JoinP p;
  p.part = part;
  p.residual = static_cast<const uint16_t*>(a.residual);
  p.bias = a.bias;
  p.y = static_cast<uint16_t*>(a.y);
  p.z = static_cast<uint16_t*>(a.z);
  p.M = a.M;
  p.N = a.N;
  p.ld = (a.N + 7) / 8 * 8;
  p.ld_residual = a.ld_residual;
  p.ld_y = a.ld_y;
  p.ld_z = a.ld_z;
  p.splits = splits;
  p.b32 = a.b_fmt == GLU_FMT_FP32;
  auto kern = a.act == GLU_ACT_SILU        ? linear_join_kernel<GLU_ACT_SILU>
              : a.act == GLU_ACT_GELU_TANH ? linear_join_kernel<GLU_ACT_GELU_TANH>
              : a.act == GLU_ACT_RELU      ? linear_join_kernel<GLU_ACT_RELU>
              : a.act == GLU_ACT_GELU_ERF  ? linear_join_kernel<GLU_ACT_GELU_ERF>
                                           : linear_join_kernel<GLU_ACT_IDENTITY>;
  return launch_kernel(kern, dim3(unsigned((a.M * ((a.N + 7) / 8) + 255) / 256)), 256, 0, s, p, true);
}

cudaError_t launch_linear_dz(int act, const DzP& q, cudaStream_t s) {
  auto kern = act == GLU_ACT_SILU        ? dz_kernel<GLU_ACT_SILU>
              : act == GLU_ACT_GELU_TANH ? dz_kernel<GLU_ACT_GELU_TANH>
              : act == GLU_ACT_RELU      ? dz_kernel<GLU_ACT_RELU>
              : act == GLU_ACT_GELU_ERF  ? dz_kernel<GLU_ACT_GELU_ERF>
                                         : dz_kernel<GLU_ACT_IDENTITY>;
  const cudaError_t e = launch_kernel(kern, dim3(unsigned(q.slots), unsigned((q.N + kDzCols - 1) / kDzCols)), dim3(32, 8), 0, s, q, true);
  if (e != cudaSuccess || q.db == nullptr) return e;
  return launch_kernel(db_kernel, dim3(unsigned((q.N + 31) / 32), unsigned(q.E)), dim3(32, 16), 0, s, q, true);
}

}  // namespace gq
