// Block norms, forward and backward (glu_block.h):
//
//   r = x + alpha * gate .* P(branch),   y = r * rstd(r) .* (w_pre + o),
//   P(b) = b * rstd(b) .* (w_post + o) or b.
//
// Both directions are a single pass over the rows.  Per element they read 2
// to 4 numbers and compute a few tens of operations, so DRAM bounds them:
// the forward moves x, branch, r and y once (8 bytes per element with a bf16
// stream), the backward r, branch, dy, dr, dx and dbranch (12 bytes).  Rows
// come through a ring of stages in shared memory, copied there in bulk, so
// that the loads of the next rows are in flight while a row's sums are joined
// across the block.  A stage is refilled after a barrier that those sums need
// anyway: by then every thread is done with the row it held.  16384 x 7168 with
// an fp32 stream and a gate takes 221 us forward (6.4 TB/s), 8191 x 8192 in
// bf16 135 us backward (5.9 TB/s).  Rows wider than 8192 hold more chunks per
// thread than registers (spilled: forward 90 to 120 bytes up to 16384 and 480 to
// 530 above, backward 260 to 310, 530 to 570 with a gate row per few rows) and
// fetch the weights for every row: 5461 x 12288 in bf16 259 us forward (2.1 TB/s)
// and 364 backward (2.2), 2048 x 32768 forward 260 (2.1).
#include "block.h"
#include "block_util.cuh"
#include "tma.cuh"

namespace gq {
namespace {

__device__ uint32_t g_err_norm;

constexpr int kMaxStages = 8;
constexpr int kSmemMost = 232448;  // shared memory per block
constexpr int kCtlBytes = 2048;    // of it, ahead of the stages

template <int N>
struct RingCtl {
  uint64_t full[kMaxStages];
  BlockSum<N> sums;
  int64_t item, row, end;  // the backward's next row to load, its item, the end of that item's rows
};
static_assert(sizeof(RingCtl<3>) <= kCtlBytes, "ring control block");

// Copy of `bytes` contiguous bytes (a multiple of 16, both addresses 16-byte
// aligned) into shared memory, completed on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Waits that gave up leave a mark and are not repeated: what follows runs on
// with whatever the stage holds, within its bounds, to its end.
struct RingWait {
  bool dead = false;
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    if (dead) return;
    if (!mbar_wait(bar, parity)) {
      dead = true;
      atomicOr(&g_err_norm, kErrWaitFull);
    }
  }
};

// The chunk in which a row's width ends (n of its columns are in it), into
// shared memory with zeros behind the width; nothing behind it is read.  Bulk
// copies take whole chunks, so this one comes apart, and every chunk is read
// alike.  (A case of its own for it at each read, with the stores below by
// single elements, took 440 us for 14566 x 4607 backward in bf16 and 208
// forward; 4608 columns take 193 and 148.)
template <typename T>
__device__ __forceinline__ void load_tail(void* dst, const T* src, int n) {
  const uint32_t d = smem_u32(dst), bytes = uint32_t(n * sizeof(T));
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes < 16 ? bytes : 16) : "memory");
  if (sizeof(T) == 4)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(d + 16), "l"(bytes > 16 ? src + 4 : src),
                 "r"(bytes > 16 ? bytes - 16 : 0)
                 : "memory");
}
// Counts one arrival when the copies of this thread so far have landed.
__device__ __forceinline__ void tails_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A chunk of eight columns (from column c) of a staged row.
template <typename T>
__device__ __forceinline__ F8 staged8(const uint8_t* stage, int c) {
  if (sizeof(T) == 2) return pairs(*reinterpret_cast<const uint4*>(stage + 2 * c));
  const float4 a = *reinterpret_cast<const float4*>(stage + 4 * c), b = *reinterpret_cast<const float4*>(stage + 4 * c + 16);
  return {{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
}
template <typename T>
__device__ __forceinline__ F8 direct8(const T* row, int c, int n) {
  float v[8];
  load8(row + c, n, v);
  return pairs(v);
}

// w + o of a chunk of a weight vector, times `scale`, times the gate's if there is one.
__device__ __forceinline__ F8 weight8(const void* w, bool f32, float o, float scale, const uint16_t* gate, int c, int n) {
  float v[8];
  if (w) {
    vec8(w, f32, c, n, o, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= scale;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = scale;
  }
  if (gate) {
    float g[8];
    vec8(gate, false, c, n, 0.0f, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= g[i];
  }
  return pairs(v);
}

// Stores a thread's chunk k of V.  RAGGED: the width may end inside the last of
// them (a row has more chunks than V - 1 per thread).
template <bool RAGGED, int V, typename T>
__device__ __forceinline__ void store_last(int k, T* p, int n, const F8& f) {
  if (RAGGED && k == V - 1) store8<true>(p, n, f);
  else store8<false>(p, n, f);
}

struct NormFwdP {
  const void* x;
  const uint16_t* branch;
  const uint16_t* gate;
  const void *w_pre, *w_post;
  void* r;
  uint16_t* y;
  float *rstd_pre, *rstd_post;
  int64_t M, D, rows_per_gate;
  int64_t ld_x, ld_branch, ld_gate, ld_r, ld_y;
  float alpha, w_offset, eps;
  int w32, stages, stage_bytes;
  int stream_gate;  // the gate's row is staged with each row (few rows share one)
};

// 1 / sqrt(sum / D + eps), with the reciprocal of D.
__device__ __forceinline__ float rstd_of(float sum, float per_d, float eps) {
  return __frcp_rn(__fsqrt_rn(fmaf(sum, per_d, eps)));
}

// Few rows: one block per row, one chunk per thread, straight from memory.
template <typename XT>
__global__ void __launch_bounds__(1024) norm_fwd_row_kernel(const NormFwdP p) {
  __shared__ BlockSum<1> sums;
  uint32_t buf = 0;
  const int D = int(p.D), c = 8 * int(threadIdx.x), threads = blockDim.x;
  const int64_t m = blockIdx.x;
  const float per_d = __frcp_rn(float(D));
  after_previous();
  next_may_come();
  F8 r = zeros(), b = zeros(), w = zeros();
  float2 s2 = make_float2(0.0f, 0.0f);
  if (c < D) {
    r = direct8(static_cast<const XT*>(p.x) + m * p.ld_x, c, D - c);
    if (p.w_pre) w = weight8(p.w_pre, p.w32, p.w_offset, 1.0f, nullptr, c, D - c);
    if (p.branch) {
      b = direct8(p.branch + m * p.ld_branch, c, D - c);
      const F8 f = weight8(p.w_post, p.w32, p.w_offset, p.alpha, p.gate ? p.gate + (m / p.rows_per_gate) * p.ld_gate : nullptr, c, D - c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s2 = fma_2(b.v[i], b.v[i], s2);
        b.v[i] = mul_2(b.v[i], f.v[i]);
      }
    }
  }
  if (p.branch) {
    float rs = 1.0f;
    if (p.w_post) {
      float s[1] = {sum2(s2)};
      block_sum(sums, buf, threads, s);
      rs = rstd_of(s[0], per_d, p.eps);
      if (threadIdx.x == 0) p.rstd_post[m] = rs;
    }
    if (c < D) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r.v[i] = fma_2(b.v[i], both(rs), r.v[i]);
      store8<true>(static_cast<XT*>(p.r) + m * p.ld_r + c, D - c, r);
    }
  }
  if (!p.w_pre) return;
  s2 = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) s2 = fma_2(r.v[i], r.v[i], s2);
  float s[1] = {sum2(s2)};
  block_sum(sums, buf, threads, s);
  const float rs = rstd_of(s[0], per_d, p.eps);
  if (threadIdx.x == 0) p.rstd_pre[m] = rs;
  if (c >= D) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = mul_2(mul_2(r.v[i], w.v[i]), both(rs));
  store8<true>(p.y + m * p.ld_y + c, D - c, r);
}

// Many rows: each block takes consecutive ones through a ring of staged rows,
// chunk k of thread t starting at column 8 (t + k * threads).  One exchange per
// row: the sum of squares of r goes with that of the next row's branch, which
// is in registers by then.  (With an exchange for each, 16384 x 7168 took 252
// us with an fp32 stream and 190 us with a bf16 one.)  Up to V = 2 chunks per thread (D <= 8192) the weights of a thread's columns
// stay in its registers, wider rows fetch them again.
template <typename XT, int V, bool RAGGED>
__global__ void __launch_bounds__(512, 1) norm_fwd_kernel(const NormFwdP p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  after_previous();
  next_may_come();
  RingCtl<2>* ctl = reinterpret_cast<RingCtl<2>*>(smem);
  uint8_t* stages = smem + kCtlBytes;
  const int threads = blockDim.x, D = int(p.D), tid = threadIdx.x;
  const uint32_t wide = uint32_t((D + 7) / 8) * 16, xb = wide / 2 * sizeof(XT), at_g = xb + (p.branch ? wide : 0u);  // a stage
  const int c_tail = D / 8 * 8;  // RAGGED: where the last chunk begins
  const int64_t m0 = p.M * blockIdx.x / gridDim.x, m1 = p.M * (blockIdx.x + 1) / gridDim.x;
  // loads row m into stage s (thread 0; RAGGED: its tails by a thread of the
  // next warp, 14566 x 4607 in fp32 184 -> 174 us)
  const int tail_tid = threads > 32 ? 32 : 0;
  auto load = [&](int64_t m, int s) {
    uint8_t* st = stages + s * p.stage_bytes;
    uint64_t* bar = &ctl->full[s];
    if (!RAGGED || tid == 0) {
      const uint32_t bytes = RAGGED ? uint32_t(c_tail) * 2 : wide, x_bytes = bytes / 2 * sizeof(XT);
      mbar_arrive_expect_tx(bar, RAGGED ? x_bytes + (p.branch ? bytes : 0u) + (p.stream_gate ? bytes : 0u) : uint32_t(p.stage_bytes));
      if (!RAGGED || bytes) {
        bulk_load(st, static_cast<const XT*>(p.x) + m * p.ld_x, x_bytes, bar);
        if (p.branch) bulk_load(st + xb, p.branch + m * p.ld_branch, bytes, bar);
        if (p.stream_gate) bulk_load(st + at_g, p.gate + m / p.rows_per_gate * p.ld_gate, bytes, bar);
      }
    }
    if (RAGGED && tid == tail_tid) {
      load_tail(st + c_tail * sizeof(XT), static_cast<const XT*>(p.x) + m * p.ld_x + c_tail, D - c_tail);
      if (p.branch) load_tail(st + xb + 2 * c_tail, p.branch + m * p.ld_branch + c_tail, D - c_tail);
      if (p.stream_gate) load_tail(st + at_g + 2 * c_tail, p.gate + m / p.rows_per_gate * p.ld_gate + c_tail, D - c_tail);
      tails_arrive(bar);
    }
  };
  const bool loads = tid == 0 || (RAGGED && tid == tail_tid);
  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(&ctl->full[s], RAGGED ? 2 : 1);
    fence_barrier_init();
  }
  if (RAGGED) __syncthreads();
  if (loads)
    for (int s = 0; s < p.stages; ++s)
      if (m0 + s < m1) load(m0 + s, s);
  __syncthreads();
  constexpr bool kHold = V <= 2;
  F8 w[kHold ? V : 1], f[kHold ? V : 1];
  if (kHold && p.w_pre) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = 8 * (tid + k * threads);
      if (c < D) w[kHold ? k : 0] = weight8(p.w_pre, p.w32, p.w_offset, 1.0f, nullptr, c, D - c);
    }
  }
  RingWait wait;
  int s = 0;  // the stage of the next row to read
  uint32_t parity = 0, buf = 0;
  const float per_d = __frcp_rn(float(D));
  int64_t grp = 0, g_end = m0;  // the gate row, and the first row past its rows
  int64_t f_end = m0;           // first row that f does not hold for
  F8 x[V], b[V];                // the row read last: the stream, and the branch times f (with the gate)
  auto read_row = [&](int64_t m) {
    if (m >= g_end) {
      grp = m / p.rows_per_gate;
      g_end = (grp + 1) * p.rows_per_gate;
    }
    const uint16_t* gate_row = p.gate + grp * p.ld_gate;
    auto factors = [&](int c) {
      return weight8(p.w_post, p.w32, p.w_offset, p.alpha, p.gate && !p.stream_gate ? gate_row : nullptr, c, D - c);
    };
    if (kHold && p.branch && m >= f_end) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = 8 * (tid + k * threads);
        if (c < D) f[kHold ? k : 0] = factors(c);
      }
      f_end = p.gate && !p.stream_gate ? g_end : m1;
    }
    const uint8_t* st = stages + s * p.stage_bytes;
    wait(&ctl->full[s], parity);
    float2 sq = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = 8 * (tid + k * threads);
      if (c >= D) continue;
      x[k] = staged8<XT>(st, c);
      if (!p.branch) continue;
      b[k] = staged8<uint16_t>(st + xb, c);
      const F8 fk = kHold ? f[kHold ? k : 0] : factors(c);
      F8 g = zeros();
      if (p.stream_gate) g = staged8<uint16_t>(st + at_g, c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sq = fma_2(b[k].v[i], b[k].v[i], sq);
        b[k].v[i] = mul_2(b[k].v[i], fk.v[i]);
        if (p.stream_gate) b[k].v[i] = mul_2(b[k].v[i], g.v[i]);
      }
    }
    return sum2(sq);
  };
  // every thread has read row m: its stage takes the row `stages` further on
  auto free_row = [&](int64_t m) {
    if (loads && m + p.stages < m1) load(m + p.stages, s);
    if (++s == p.stages) s = 0, parity ^= 1u;
  };
  XT* r_out = static_cast<XT*>(p.r) + m0 * p.ld_r;
  uint16_t* y_out = p.y + m0 * p.ld_y;
  float sum[2] = {0.0f, 0.0f};
  for (int64_t m = m0 - 1; m < m1; ++m) {  // row m is written, row m + 1 read
    const bool row = m >= m0;
    F8 r[V];
    float2 s2 = make_float2(0.0f, 0.0f);
    if (row) {
      const float rq = p.w_post ? rstd_of(sum[1], per_d, p.eps) : 1.0f;
      if (p.w_post && tid == 0) p.rstd_post[m] = rq;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = 8 * (tid + k * threads);
        if (c >= D) continue;
        r[k] = x[k];
        if (p.branch) {
#pragma unroll
          for (int i = 0; i < 4; ++i) r[k].v[i] = fma_2(b[k].v[i], both(rq), r[k].v[i]);
          store_last<RAGGED, V>(k, r_out + c, D - c, r[k]);
        }
        if (!p.w_pre) continue;
        const F8 wk = kHold ? w[kHold ? k : 0] : weight8(p.w_pre, p.w32, p.w_offset, 1.0f, nullptr, c, D - c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s2 = fma_2(r[k].v[i], r[k].v[i], s2);
          r[k].v[i] = mul_2(r[k].v[i], wk.v[i]);
        }
      }
      r_out += p.ld_r;
    }
    sum[0] = sum2(s2);
    sum[1] = m + 1 < m1 ? read_row(m + 1) : 0.0f;
    block_sum(ctl->sums, buf, threads, sum);
    if (m + 1 < m1) free_row(m + 1);
    if (!row || !p.w_pre) continue;
    const float rs = rstd_of(sum[0], per_d, p.eps);
    if (tid == 0) p.rstd_pre[m] = rs;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = 8 * (tid + k * threads);
      if (c >= D) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) r[k].v[i] = mul_2(r[k].v[i], both(rs));
      store_last<RAGGED, V>(k, y_out + c, D - c, r[k]);
    }
    y_out += p.ld_y;
  }
}

int row_threads(int64_t chunks, int V) { return int(((chunks + V - 1) / V + 31) / 32 * 32); }
int row_chunks(int64_t chunks) { return chunks <= 32 ? 1 : chunks <= 1024 ? 2 : chunks <= 2048 ? 4 : 8; }  // per thread

// The ring's stages for `blocks` blocks per SM.
int ring_stages(int stage_bytes, int blocks) {
  const int room = (blocks == 1 ? kSmemMost : 228 * 1024 / blocks - 1024) - kCtlBytes;
  const int n = stage_bytes == 0 ? 1 : room / stage_bytes;
  return n > kMaxStages ? kMaxStages : n < 1 ? 1 : n;
}
// Blocks per SM: 512 threads with 128 registers each.
int ring_blocks(int threads) { return 512 / threads; }

template <typename XT, int V>
cudaError_t launch_fwd_rows(NormFwdP p, cudaStream_t s, const DevInfo& d) {
  const int threads = row_threads((p.D + 7) / 8, V), blocks = ring_blocks(threads);
  // a gate row shared by few rows comes with each (where one stage has room
  // for it), else its factors are fetched when it changes
  const int64_t wide = (p.D + 7) / 8 * 8;
  p.stream_gate = p.gate != nullptr && p.rows_per_gate < 16 && wide * int64_t(sizeof(XT) + 4) + kCtlBytes <= kSmemMost;
  p.stage_bytes = int(wide * (sizeof(XT) + (p.branch ? 2 : 0) + (p.stream_gate ? 2 : 0)));
  p.stages = ring_stages(p.stage_bytes, blocks);
  const int smem = kCtlBytes + p.stages * p.stage_bytes;
  if (smem > kSmemMost) return cudaErrorInvalidValue;
  auto kern = p.D % 8 != 0 ? norm_fwd_kernel<XT, V, true> : norm_fwd_kernel<XT, V, false>;
  static SmemLimit limit[2];
  const cudaError_t e = limit[p.D % 8 != 0].raise(reinterpret_cast<const void*>(kern), kSmemMost);
  if (e != cudaSuccess) return e;
  const int64_t most = int64_t(d.sms) * blocks;
  return launch_kernel(kern, int(p.M < most ? p.M : most), threads, smem, s, p, true);
}

template <typename XT>
cudaError_t launch_fwd_t(const NormFwdP& p, cudaStream_t s, const DevInfo& d) {
  const int64_t chunks = (p.D + 7) / 8;
  if (p.M <= 2 * d.sms && chunks <= 1024) return launch_kernel(norm_fwd_row_kernel<XT>, int(p.M), row_threads(chunks, 1), 0, s, p, true);
  switch (row_chunks(chunks)) {
    case 1: return launch_fwd_rows<XT, 1>(p, s, d);
    case 2: return launch_fwd_rows<XT, 2>(p, s, d);
    case 4: return launch_fwd_rows<XT, 4>(p, s, d);
    default: return launch_fwd_rows<XT, 8>(p, s, d);
  }
}

// ------------------------------------------------------------- backward --

struct NormBwdP {
  const void *r, *dr;
  const uint16_t *branch, *gate, *dy;
  const void *w_pre, *w_post;
  const float *rstd_pre, *rstd_post;
  void* dx;
  uint16_t* dbranch;
  float* part_pre;   // [gridDim.x, D]
  float* part_x;     // [items, D], or NULL
  float* part_post;  // [gridDim.x, D], or NULL
  float* dgate;      // written here where an item is a whole gate row's rows
  int64_t M, D, rows_per_gate, pieces, items;  // an item: one of `pieces` parts of a gate row's rows
  int64_t ld_r, ld_dr, ld_branch, ld_gate, ld_dy, ld_dx, ld_dbranch;
  float alpha, w_offset;
  int w32, stages, stage_bytes;
};

// A chunk of sums, [.., D] contiguous: rows start on 16 bytes unless RAGGED.
template <bool RAGGED>
__device__ __forceinline__ void store_sums(float* row, int c, int D, const F8& v) {
  if (!RAGGED) {
    store8<false>(row + c, 8, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < D) row[c + i] = (i & 1) ? v.v[i / 2].y : v.v[i / 2].x;
  }
}

// A thread has the same columns of every row of its block, so the sums over
// rows stay in its registers.  With w = w_pre + o, h = alpha gate (w_post + o)
// (or alpha gate), t = dr + rstd_pre dy w and b = branch:
//   dR = t - r rstd_pre^2 S1 / D,                     S1 = sum rstd_pre dy w r
//   dbranch = rstd_post h dR - b rstd_post^2 S / D,   S = sum h dR rstd_post b
// S is had with S1 in one exchange across the block:
//   S = rstd_post (S2 - rstd_pre^2 (S1 / D) S3),  S2 = sum h b t,  S3 = sum h b r.
// dw_pre sums dy r rstd_pre.  dgate and dw_post are both multiples of X = sum
// over the rows of one gate row of dR b rstd_post: dgate = alpha (w_post + o)
// X, dw_post = sum over gate rows of alpha gate X.  A block takes whole items
// (consecutive rows that share a gate row).  MANY: an item is all the rows of
// a gate row, the gate's row is staged with them, and the block finishes dgate
// and sums dw_post itself; else X goes out per item and the join does both.
//
// At 8191 x 8192 (bf16) one block of 16 warps per SM has three 64 KB stages:
// two rows in flight while one is worked on.
template <typename XT, int V, bool MANY, bool RAGGED>
__global__ void __launch_bounds__(512, 1) norm_bwd_kernel(const NormBwdP p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  after_previous();
  next_may_come();
  RingCtl<3>* ctl = reinterpret_cast<RingCtl<3>*>(smem);
  uint8_t* stages = smem + kCtlBytes;
  const int threads = blockDim.x, D = int(p.D), tid = threadIdx.x;
  const uint32_t wide = uint32_t((D + 7) / 8) * 16, xb = wide / 2 * sizeof(XT);
  const int c_tail = D / 8 * 8;  // RAGGED: where the last chunk begins
  const bool pre = p.w_pre != nullptr, post = p.w_post != nullptr, br = p.branch != nullptr, has_dr = p.dr != nullptr;
  // a stage: r, dy (pre), dr (given), branch (given), gate (MANY)
  const uint32_t at_dy = pre ? xb : 0u, at_dr = at_dy + (pre ? wide : 0u), at_b = at_dr + (has_dr ? xb : 0u), at_g = at_b + wide;
  // loads the next row of this block's items into stage s, if there is one (one
  // thread, the tails too: a second one for those changed the times by -3 to 3 %)
  auto load_next = [&](int s) {
    while (ctl->row >= ctl->end) {
      if (ctl->item >= p.items) return;
      const int64_t base = ctl->item / p.pieces * p.rows_per_gate, piece = ctl->item % p.pieces;
      ctl->row = base + piece * p.rows_per_gate / p.pieces;
      ctl->end = base + (piece + 1) * p.rows_per_gate / p.pieces;
      ctl->item += gridDim.x;
    }
    const int64_t m = ctl->row++;
    uint8_t* st = stages + s * p.stage_bytes;
    uint64_t* bar = &ctl->full[s];
    const XT *r = static_cast<const XT*>(p.r) + m * p.ld_r, *dr = static_cast<const XT*>(p.dr) + m * p.ld_dr;
    const uint16_t *dy = p.dy + m * p.ld_dy, *b = p.branch + m * p.ld_branch, *g = MANY ? p.gate + m / p.rows_per_gate * p.ld_gate : nullptr;
    const uint32_t bytes = RAGGED ? uint32_t(c_tail) * 2 : wide, x_bytes = bytes / 2 * sizeof(XT);
    mbar_arrive_expect_tx(bar, (pre ? x_bytes + bytes : 0u) + (has_dr ? x_bytes : 0u) + (br ? bytes : 0u) + (MANY ? bytes : 0u));
    if (!RAGGED || bytes) {
      if (pre) bulk_load(st, r, x_bytes, bar), bulk_load(st + at_dy, dy, bytes, bar);
      if (has_dr) bulk_load(st + at_dr, dr, x_bytes, bar);
      if (br) bulk_load(st + at_b, b, bytes, bar);
      if (MANY) bulk_load(st + at_g, g, bytes, bar);
    }
    if (RAGGED) {
      const int n = D - c_tail;
      if (pre) load_tail(st + x_bytes, r + c_tail, n), load_tail(st + at_dy + bytes, dy + c_tail, n);
      if (has_dr) load_tail(st + at_dr + x_bytes, dr + c_tail, n);
      if (br) load_tail(st + at_b + bytes, b + c_tail, n);
      if (MANY) load_tail(st + at_g + bytes, g + c_tail, n);
      tails_arrive(bar);
    }
  };
  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(&ctl->full[s], RAGGED ? 2 : 1);
    fence_barrier_init();
    ctl->item = blockIdx.x;
    ctl->row = ctl->end = 0;
    for (int s = 0; s < p.stages; ++s) load_next(s);
  }
  __syncthreads();
  F8 a_pre[V], a_x[V], a_post[MANY ? V : 1];
#pragma unroll
  for (int k = 0; k < V; ++k) a_pre[k] = a_x[k] = a_post[MANY ? k : 0] = zeros();
  // w and h (MANY: without the gate) of this thread's columns: in registers for
  // up to two chunks, fetched again for every row otherwise
  constexpr bool kHold = V <= 2;
  F8 w[kHold ? V : 1], h[kHold ? V : 1];
  auto fetch_w = [&](int c) { return weight8(p.w_pre, p.w32, p.w_offset, 1.0f, nullptr, c, D - c); };
  auto fetch_h = [&](int64_t grp, int c) {
    return weight8(p.w_post, p.w32, p.w_offset, p.alpha, !MANY && p.gate ? p.gate + grp * p.ld_gate : nullptr, c, D - c);
  };
  if (kHold) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = 8 * (tid + k * threads);
      if (c < D && pre) w[kHold ? k : 0] = fetch_w(c);
      if (c < D && br && MANY) h[kHold ? k : 0] = fetch_h(0, c);
    }
  }
  const float per_d = __frcp_rn(float(D));
  RingWait wait;
  int s = 0, last = -1;  // the stage of the row before this one
  uint32_t parity = 0, buf = 0;
  for (int64_t it = blockIdx.x; it < p.items; it += gridDim.x) {
    const int64_t grp = it / p.pieces, base = grp * p.rows_per_gate, piece = it % p.pieces;
    const int64_t m1 = base + (piece + 1) * p.rows_per_gate / p.pieces;
    if (kHold && br && !MANY) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = 8 * (tid + k * threads);
        if (c < D) h[kHold ? k : 0] = fetch_h(grp, c);
      }
    }
    const int64_t m0 = base + piece * p.rows_per_gate / p.pieces;
    XT* dx = static_cast<XT*>(p.dx) + m0 * p.ld_dx;
    uint16_t* db = p.dbranch + m0 * p.ld_dbranch;
    float rs32 = 0.0f, rp32 = 1.0f;  // lane l: the rstd of the l-th of 32 rows, loaded together
    for (int64_t m = m0; m < m1; ++m, dx += p.ld_dx, db += p.ld_dbranch) {
      const uint8_t* st = stages + s * p.stage_bytes;
      const int row32 = int(m - m0) & 31;
      if (row32 == 0) {
        const int64_t ml = m + (tid & 31);
        if (pre && ml < m1) rs32 = p.rstd_pre[ml];
        if (post && ml < m1) rp32 = p.rstd_post[ml];
      }
      const float rs = __shfl_sync(0xFFFFFFFFu, rs32, row32), rp = __shfl_sync(0xFFFFFFFFu, rp32, row32);
      auto h_of = [&](int k, int c) {
        F8 f = kHold ? h[kHold ? k : 0] : fetch_h(grp, c);
        if (MANY) {
          const F8 g = staged8<uint16_t>(st + at_g, c);
#pragma unroll
          for (int i = 0; i < 4; ++i) f.v[i] = mul_2(f.v[i], g.v[i]);
        }
        return f;
      };
      wait(&ctl->full[s], parity);
      F8 t[V];
      float2 s1 = make_float2(0.0f, 0.0f), s2 = s1, s3 = s1;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = 8 * (tid + k * threads);
        if (c >= D) continue;
        t[k] = has_dr ? staged8<XT>(st + at_dr, c) : zeros();
        F8 r = zeros();
        if (pre) {
          r = staged8<XT>(st, c);
          F8 v = staged8<uint16_t>(st + at_dy, c);
          const F8 wk = kHold ? w[kHold ? k : 0] : fetch_w(c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v.v[i] = mul_2(v.v[i], both(rs));
            a_pre[k].v[i] = fma_2(v.v[i], r.v[i], a_pre[k].v[i]);
            v.v[i] = mul_2(v.v[i], wk.v[i]);
            s1 = fma_2(v.v[i], r.v[i], s1);
            t[k].v[i] = add_2(v.v[i], t[k].v[i]);
          }
        }
        if (post) {
          const F8 b = staged8<uint16_t>(st + at_b, c), hk = h_of(k, c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 q = mul_2(b.v[i], hk.v[i]);
            s2 = fma_2(q, t[k].v[i], s2);
            if (pre) s3 = fma_2(q, r.v[i], s3);
          }
        }
      }
      float sum[3] = {sum2(s1), sum2(s2), sum2(s3)};
      if (pre || post) block_sum(ctl->sums, buf, threads, sum);
      else row_barrier(threads);
      // every thread is done with the row before this one
      if (tid == 0 && last >= 0) load_next(last);
      // The sums come first: with rows of 1e14 or 1e-14 the powers of an rstd
      // alone are outside fp32's range, their products with the sums are not.
      const float k1 = -(sum[0] * per_d * rs) * rs;
      const float k2 = -(fmaf(k1, sum[2], sum[1]) * rp * per_d * rp) * rp;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = 8 * (tid + k * threads);
        if (c >= D) continue;
        if (pre) {
          const F8 r = staged8<XT>(st, c);
#pragma unroll
          for (int i = 0; i < 4; ++i) t[k].v[i] = fma_2(r.v[i], both(k1), t[k].v[i]);
        }
        store_last<RAGGED, V>(k, dx + c, D - c, t[k]);
        if (!br) continue;
        F8 b = staged8<uint16_t>(st + at_b, c);
        const F8 hk = h_of(k, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 e = post ? mul_2(t[k].v[i], both(rp)) : t[k].v[i];
          a_x[k].v[i] = fma_2(e, b.v[i], a_x[k].v[i]);
          b.v[i] = post ? fma_2(b.v[i], both(k2), mul_2(e, hk.v[i])) : mul_2(e, hk.v[i]);
        }
        store_last<RAGGED, V>(k, db + c, D - c, b);
      }
      if (MANY && m + 1 == m1) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const int c = 8 * (tid + k * threads);
          if (c >= D) continue;
          const F8 g = staged8<uint16_t>(st + at_g, c);
          F8 out = kHold ? h[kHold ? k : 0] : fetch_h(grp, c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a_post[MANY ? k : 0].v[i] = fma_2(mul_2(g.v[i], both(p.alpha)), a_x[k].v[i], a_post[MANY ? k : 0].v[i]);
            out.v[i] = mul_2(out.v[i], a_x[k].v[i]);
          }
          store_sums<RAGGED>(p.dgate + grp * D, c, D, out);
          a_x[k] = zeros();
        }
      }
      last = s;
      if (p.stages == 1) {  // a row's load follows the row before it
        row_barrier(threads);
        if (tid == 0) load_next(0);
        last = -1;
      }
      if (++s == p.stages) s = 0, parity ^= 1u;
    }
    if (!MANY && p.part_x) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = 8 * (tid + k * threads);
        if (c < D) store_sums<RAGGED>(p.part_x + it * D, c, D, a_x[k]);
        a_x[k] = zeros();
      }
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = 8 * (tid + k * threads);
    if (c >= D) continue;
    if (pre) store_sums<RAGGED>(p.part_pre + int64_t(blockIdx.x) * D, c, D, a_pre[k]);
    if (MANY && post) store_sums<RAGGED>(p.part_post + int64_t(blockIdx.x) * D, c, D, a_post[MANY ? k : 0]);
  }
}

// The sums over blocks and items, in a fixed order: 32 columns per block, 32
// threads per column, eight loads of each in flight.  (part_x has few items,
// at most four per block: divided in 64 bits their numbers took 11 us of 2000 x
// 1024's 33.)  blockIdx.y: dw_pre, dw_post, then the gate rows.
struct JoinP {
  const float *part_pre, *part_post, *part_x;
  const uint16_t* gate;
  const void* w_post;
  float *dw_pre, *dw_post, *dgate;
  int64_t D, ld_gate, items, pieces;
  int blocks, w32;
  float alpha, w_offset;
};
__global__ void __launch_bounds__(1024) join_kernel(const JoinP p) {
  __shared__ float sh[32][33];
  int64_t y = blockIdx.y;
  const int64_t c = int64_t(blockIdx.x) * 32 + threadIdx.x;
  int what = 2;  // 0: dw_pre, 1: dw_post, 2: gate row y
  after_previous();
  next_may_come();
  if (p.dw_pre) what = y-- == 0 ? 0 : 2;
  if (what == 2 && p.dw_post) what = y-- == 0 ? 1 : 2;
  float v = 0.0f;
  if (c < p.D) {
    if (what == 2) {
#pragma unroll 8
      for (int64_t i = threadIdx.y; i < p.pieces; i += 32) v += p.part_x[(y * p.pieces + i) * p.D + c];
    } else if (what == 1 && p.part_x) {
#pragma unroll 8
      for (uint32_t i = threadIdx.y; i < uint32_t(p.items); i += 32) {
        const float x = p.part_x[i * p.D + c];
        v = p.gate ? fmaf(bf16_of_bits(p.gate[i / uint32_t(p.pieces) * p.ld_gate + c]), x, v) : v + x;
      }
    } else {
      const float* q = what == 0 ? p.part_pre : p.part_post;
#pragma unroll 8
      for (int64_t i = threadIdx.y; i < p.blocks; i += 32) v += q[i * p.D + c];
    }
  }
  sh[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0 || c >= p.D) return;
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) v += sh[i][threadIdx.x];
  if (what == 0) {
    p.dw_pre[c] = v;
  } else if (what == 1) {
    p.dw_post[c] = p.part_x ? p.alpha * v : v;
  } else {
    float w = p.alpha;
    if (p.w_post)
      w *= (p.w32 ? static_cast<const float*>(p.w_post)[c] : bf16_of_bits(static_cast<const uint16_t*>(p.w_post)[c])) + p.w_offset;
    p.dgate[y * p.D + c] = w * v;
  }
}

// The backward's split, a function of the shape alone (for GB300's 152 SMs).
struct NormBwdPlan {
  int V, threads, per_sm, grid;
  int64_t pieces, items;
  bool many;
};
NormBwdPlan norm_bwd_plan(int64_t M, int64_t D, int64_t gates) {
  NormBwdPlan q;
  const int64_t chunks = (D + 7) / 8;
  q.V = row_chunks(chunks);
  q.threads = row_threads(chunks, q.V);
  q.per_sm = ring_blocks(q.threads);
  const int64_t blocks = 152 * q.per_sm;
  const int64_t groups = gates > 0 ? gates : 1, rows = M / groups;
  // parts per gate row: the choice among those of 1 to 4 items per block
  // with the fewest rows on the busiest block
  q.pieces = 1;
  int64_t best = -1;
  for (int64_t k = 1; k <= 4; ++k) {
    int64_t c = k * blocks / groups;
    c = c < 1 ? 1 : c > rows ? rows : c;
    const int64_t busiest = (groups * c + blocks - 1) / blocks * ((rows + c - 1) / c);
    if (best < 0 || busiest < best) best = busiest, q.pieces = c;
  }
  q.items = groups * q.pieces;
  q.grid = int(q.items < blocks ? q.items : blocks);
  q.many = gates > 1 && q.pieces == 1;
  return q;
}

template <typename XT, int V, bool MANY>
cudaError_t launch_bwd_v(NormBwdP p, const NormBwdPlan& q, cudaStream_t s) {
  p.stage_bytes =
      int((p.D + 7) / 8 * 8 * ((p.w_pre ? sizeof(XT) + 2 : 0) + (p.dr ? sizeof(XT) : 0) + (p.branch ? 2 : 0) + (MANY ? 2 : 0)));
  p.stages = ring_stages(p.stage_bytes, q.per_sm);
  const int smem = kCtlBytes + p.stages * p.stage_bytes;
  if (smem > kSmemMost) return cudaErrorInvalidValue;
  auto kern = p.D % 8 != 0 ? norm_bwd_kernel<XT, V, MANY, true> : norm_bwd_kernel<XT, V, MANY, false>;
  static SmemLimit limit[2];
  const cudaError_t e = limit[p.D % 8 != 0].raise(reinterpret_cast<const void*>(kern), kSmemMost);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, q.grid, q.threads, smem, s, p, true);
}

template <typename XT, bool MANY>
cudaError_t launch_bwd_t(const NormBwdP& p, const NormBwdPlan& q, cudaStream_t s) {
  switch (q.V) {
    case 1: return launch_bwd_v<XT, 1, MANY>(p, q, s);
    case 2: return launch_bwd_v<XT, 2, MANY>(p, q, s);
    default: return launch_bwd_v<XT, 4, MANY>(p, q, s);
  }
}

}  // namespace

cudaError_t launch_norm_fwd(const glu_block_norm_fwd_args& a, cudaStream_t s, const DevInfo& d) {
  NormFwdP p = {};
  p.x = a.x;
  p.branch = static_cast<const uint16_t*>(a.branch);
  p.gate = static_cast<const uint16_t*>(a.gate);
  p.w_pre = a.w_pre;
  p.w_post = a.w_post;
  p.r = a.r;
  p.y = static_cast<uint16_t*>(a.y);
  p.rstd_pre = a.rstd_pre;
  p.rstd_post = a.rstd_post;
  p.M = a.M;
  p.D = a.D;
  p.rows_per_gate = a.gates > 0 ? a.M / a.gates : a.M;
  p.ld_x = a.ld_x;
  p.ld_branch = a.ld_branch;
  p.ld_gate = a.ld_gate;
  p.ld_r = a.ld_r;
  p.ld_y = a.ld_y;
  p.alpha = a.alpha;
  p.w_offset = a.w_offset;
  p.eps = a.eps;
  p.w32 = a.w_fmt == GLU_FMT_FP32;
  return a.x_fmt == GLU_FMT_FP32 ? launch_fwd_t<float>(p, s, d) : launch_fwd_t<uint16_t>(p, s, d);
}

size_t norm_bwd_workspace(int64_t M, int64_t D, int64_t gates) {
  const NormBwdPlan q = norm_bwd_plan(M, D, gates);
  return size_t(D) * 4 * (size_t(q.grid) + size_t(q.many ? q.grid : q.items));
}

cudaError_t launch_norm_bwd(const glu_block_norm_bwd_args& a, cudaStream_t s) {
  const NormBwdPlan q = norm_bwd_plan(a.M, a.D, a.gates);
  NormBwdP p = {};
  p.r = a.r;
  p.dr = a.dr;
  p.branch = static_cast<const uint16_t*>(a.branch);
  p.gate = static_cast<const uint16_t*>(a.gate);
  p.dy = static_cast<const uint16_t*>(a.dy);
  p.w_pre = a.w_pre;
  p.w_post = a.w_post;
  p.rstd_pre = a.rstd_pre;
  p.rstd_post = a.rstd_post;
  p.dx = a.dx;
  p.dbranch = static_cast<uint16_t*>(a.dbranch);
  p.part_pre = static_cast<float*>(a.workspace);
  float* second = p.part_pre + int64_t(q.grid) * a.D;
  if (q.many) p.part_post = second;
  else if (a.dw_post || a.dgate) p.part_x = second;
  p.dgate = a.dgate;
  p.M = a.M;
  p.D = a.D;
  p.rows_per_gate = a.gates > 0 ? a.M / a.gates : a.M;
  p.pieces = q.pieces;
  p.items = q.items;
  p.ld_r = a.ld_r;
  p.ld_dr = a.ld_dr;
  p.ld_branch = a.ld_branch;
  p.ld_gate = a.ld_gate;
  p.ld_dy = a.ld_dy;
  p.ld_dx = a.ld_dx;
  p.ld_dbranch = a.ld_dbranch;
  p.alpha = a.alpha;
  p.w_offset = a.w_offset;
  p.w32 = a.w_fmt == GLU_FMT_FP32;
  const cudaError_t e = a.x_fmt == GLU_FMT_FP32 ? (q.many ? launch_bwd_t<float, true>(p, q, s) : launch_bwd_t<float, false>(p, q, s))
                                                : (q.many ? launch_bwd_t<uint16_t, true>(p, q, s) : launch_bwd_t<uint16_t, false>(p, q, s));
  if (e != cudaSuccess) return e;
  JoinP j = {};
  j.part_pre = p.part_pre;
  j.part_post = p.part_post;
  j.part_x = p.part_x;
  j.gate = p.gate;
  j.w_post = a.w_post;
  j.dw_pre = a.dw_pre;
  j.dw_post = a.dw_post;
  j.dgate = q.many ? nullptr : a.dgate;
  j.D = a.D;
  j.ld_gate = a.ld_gate;
  j.items = q.items;
  j.pieces = q.pieces;
  j.blocks = q.grid;
  j.w32 = p.w32;
  j.alpha = a.alpha;
  j.w_offset = a.w_offset;
  const int64_t rows = (a.dw_pre ? 1 : 0) + (a.dw_post ? 1 : 0) + (j.dgate ? a.gates : 0);
  if (rows == 0) return cudaSuccess;
  return launch_kernel(join_kernel, dim3(unsigned((a.D + 31) / 32), unsigned(rows)), dim3(32, 32), 0, s, j, true);
}

cudaError_t read_err_norm(uint32_t* v, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(v, g_err_norm, sizeof(uint32_t));
  if (e == cudaSuccess && clear) {
    const uint32_t z = 0;
    e = cudaMemcpyToSymbol(g_err_norm, &z, sizeof(uint32_t));
  }
  return e;
}

}  // namespace gq
