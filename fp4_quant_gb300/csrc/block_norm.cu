// Block norms, forward and backward (glu_block.h):
//
//   r = x + alpha * gate .* P(branch),   y = r * rstd(r) .* (w_pre + o),
//   P(b) = b * rstd(b) .* (w_post + o) or b.
//
// Both directions are a single pass over the rows.  Per element they read 2
// to 4 numbers and compute a few tens of operations, so DRAM bounds them:
// the forward moves x, branch, r and y once (8 bytes per element with a bf16
// stream), the backward r, branch, dy, dr, dx and dbranch (12 bytes).  A row
// stays in the registers of one block between its statistics and its
// outputs.
#include "block.h"
#include "block_util.cuh"

namespace gq {
namespace {

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
  int w32;
};

__device__ __forceinline__ float rstd_of(float sum, int64_t D, float eps) {
  return __frcp_rn(__fsqrt_rn(__fdiv_rn(sum, float(D)) + eps));
}

// One block per row (grid-stride over the rows), V chunks of eight columns
// per thread: chunk k of thread t starts at column 8 (t + k * threads).
template <typename XT, int V>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const NormFwdP p) {
  __shared__ BlockSum<1> sums;
  uint32_t buf = 0;
  const int D = int(p.D);
  for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
    float r[V][8], b[V][8];
    const XT* xr = static_cast<const XT*>(p.x) + m * p.ld_x;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = 8 * int(threadIdx.x + k * blockDim.x);
      if (c < D) {
        load8(xr + c, D - c, r[k]);
        if (p.branch) load8(p.branch + m * p.ld_branch + c, D - c, b[k]);
      }
    }
    if (p.branch) {
      if (p.w_post) {
        float s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < V; ++k) {
          if (8 * int(threadIdx.x + k * blockDim.x) >= D) continue;
#pragma unroll
          for (int i = 0; i < 8; ++i) s[0] = fmaf(b[k][i], b[k][i], s[0]);
        }
        block_sum(sums, buf, s);
        const float rs = rstd_of(s[0], p.D, p.eps);
        if (threadIdx.x == 0) p.rstd_post[m] = rs;
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const int c = 8 * int(threadIdx.x + k * blockDim.x);
          if (c >= D) continue;
          float w[8];
          vec8(p.w_post, p.w32, c, D - c, p.w_offset, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) b[k][i] = b[k][i] * rs * w[i];
        }
      }
      XT* rr = static_cast<XT*>(p.r) + m * p.ld_r;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = 8 * int(threadIdx.x + k * blockDim.x);
        if (c >= D) continue;
        if (p.gate) {
          float g[8];
          vec8(p.gate + (m / p.rows_per_gate) * p.ld_gate, false, c, D - c, 0.0f, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) b[k][i] *= g[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) r[k][i] = i < D - c ? fmaf(p.alpha, b[k][i], r[k][i]) : 0.0f;
        store8(rr + c, D - c, r[k]);
      }
    }
    if (p.w_pre) {
      float s[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < V; ++k) {
        if (8 * int(threadIdx.x + k * blockDim.x) >= D) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] = fmaf(r[k][i], r[k][i], s[0]);
      }
      block_sum(sums, buf, s);
      const float rs = rstd_of(s[0], p.D, p.eps);
      if (threadIdx.x == 0) p.rstd_pre[m] = rs;
      uint16_t* yr = p.y + m * p.ld_y;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = 8 * int(threadIdx.x + k * blockDim.x);
        if (c >= D) continue;
        float w[8];
        vec8(p.w_pre, p.w32, c, D - c, p.w_offset, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = r[k][i] * rs * w[i];
        store8(yr + c, D - c, w);
      }
    }
  }
}

template <typename XT>
cudaError_t launch_fwd_t(const NormFwdP& p, cudaStream_t s, const DevInfo& d) {
  const int64_t chunks = (p.D + 7) / 8;
  // chunks per thread: one where there are fewer rows than the SMs hold
  // blocks (the row's latency counts), else blocks of about 256 threads
  const int V = chunks > 1024 ? 4 : (p.M <= 2 * d.sms || chunks <= 256) ? 1 : chunks <= 512 ? 2 : 4;
  const int threads = int(((chunks + V - 1) / V + 31) / 32 * 32);
  const int64_t most = int64_t(d.sms) * (threads > 512 ? 2 : 2048 / threads > 32 ? 32 : 2048 / threads);
  const int grid = int(p.M < most ? p.M : most);
  switch (V) {
    case 1: return launch_kernel(norm_fwd_kernel<XT, 1>, grid, threads, 0, s, p);
    case 2: return launch_kernel(norm_fwd_kernel<XT, 2>, grid, threads, 0, s, p);
    default: return launch_kernel(norm_fwd_kernel<XT, 4>, grid, threads, 0, s, p);
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
  float *part_pre, *part_post;  // [gridDim.x, D]
  float* part_gate;             // [items, D] (dgate itself where a gate row is one item)
  int64_t M, D, rows_per_gate, pieces, items;  // an item: one of `pieces` parts of a gate row's rows
  int64_t ld_r, ld_dr, ld_branch, ld_gate, ld_dy, ld_dx, ld_dbranch;
  float alpha, w_offset;
  int w32;
};

// Sums over the rows are kept in registers: a thread has the same columns of
// every row of its block.  A block takes whole items (consecutive rows that
// share a gate row), so dgate's partial sums never mix gate rows.
template <typename XT, int V>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormBwdP p) {
  __shared__ BlockSum<1> sums;
  uint32_t buf = 0;
  const int D = int(p.D);
  float a_pre[V][8], a_post[V][8], a_gate[V][8];
#pragma unroll
  for (int k = 0; k < V; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) a_pre[k][i] = a_post[k][i] = a_gate[k][i] = 0.0f;
  for (int64_t it = blockIdx.x; it < p.items; it += gridDim.x) {
    const int64_t grp = it / p.pieces, piece = it % p.pieces;
    const int64_t m0 = grp * p.rows_per_gate + piece * p.rows_per_gate / p.pieces;
    const int64_t m1 = grp * p.rows_per_gate + (piece + 1) * p.rows_per_gate / p.pieces;
    for (int64_t m = m0; m < m1; ++m) {
      float dR[V][8], n[V][8], u[V][8];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = 8 * int(threadIdx.x + k * blockDim.x);
#pragma unroll
        for (int i = 0; i < 8; ++i) dR[k][i] = 0.0f;
        if (c < D && p.dr) load8(static_cast<const XT*>(p.dr) + m * p.ld_dr + c, D - c, dR[k]);
      }
      if (p.w_pre) {
        const float rs = p.rstd_pre[m];
        float s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const int c = 8 * int(threadIdx.x + k * blockDim.x);
          if (c >= D) continue;
          float w[8];
          load8(static_cast<const XT*>(p.r) + m * p.ld_r + c, D - c, n[k]);
          load8(p.dy + m * p.ld_dy + c, D - c, u[k]);
          vec8(p.w_pre, p.w32, c, D - c, p.w_offset, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            n[k][i] *= rs;
            a_pre[k][i] = fmaf(u[k][i], n[k][i], a_pre[k][i]);
            u[k][i] *= w[i];
            s[0] = fmaf(u[k][i], n[k][i], s[0]);
          }
        }
        block_sum(sums, buf, s);
        const float mean = __fdiv_rn(s[0], float(D));
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (8 * int(threadIdx.x + k * blockDim.x) < D) {
#pragma unroll
            for (int i = 0; i < 8; ++i) dR[k][i] = fmaf(rs, fmaf(-n[k][i], mean, u[k][i]), dR[k][i]);
          }
      }
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = 8 * int(threadIdx.x + k * blockDim.x);
        if (c < D) store8(static_cast<XT*>(p.dx) + m * p.ld_dx + c, D - c, dR[k]);
      }
      if (!p.branch) continue;
      const float rs = p.w_post ? p.rstd_post[m] : 1.0f;
      float s[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = 8 * int(threadIdx.x + k * blockDim.x);
        if (c >= D) continue;
        float w[8], g[8];
        load8(p.branch + m * p.ld_branch + c, D - c, n[k]);
        if (p.w_post) vec8(p.w_post, p.w32, c, D - c, p.w_offset, w);
        if (p.gate) vec8(p.gate + grp * p.ld_gate, false, c, D - c, 0.0f, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float ad = p.alpha * dR[k][i];
          n[k][i] *= rs;
          if (p.gate) a_gate[k][i] = fmaf(ad, p.w_post ? n[k][i] * w[i] : n[k][i], a_gate[k][i]);
          u[k][i] = p.gate ? ad * g[i] : ad;  // d
          if (p.w_post) {
            a_post[k][i] = fmaf(u[k][i], n[k][i], a_post[k][i]);
            u[k][i] *= w[i];
            s[0] = fmaf(u[k][i], n[k][i], s[0]);
          }
        }
      }
      float mean = 0.0f;
      if (p.w_post) {
        block_sum(sums, buf, s);
        mean = __fdiv_rn(s[0], float(D));
      }
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = 8 * int(threadIdx.x + k * blockDim.x);
        if (c >= D) continue;
        if (p.w_post) {
#pragma unroll
          for (int i = 0; i < 8; ++i) u[k][i] = rs * fmaf(-n[k][i], mean, u[k][i]);
        }
        store8(p.dbranch + m * p.ld_dbranch + c, D - c, u[k]);
      }
    }
    if (p.gate) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = 8 * int(threadIdx.x + k * blockDim.x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (c + i < D) p.part_gate[it * D + c + i] = a_gate[k][i];
          a_gate[k][i] = 0.0f;
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = 8 * int(threadIdx.x + k * blockDim.x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (c + i >= D) continue;
      if (p.w_pre) p.part_pre[int64_t(blockIdx.x) * D + c + i] = a_pre[k][i];
      if (p.w_post) p.part_post[int64_t(blockIdx.x) * D + c + i] = a_post[k][i];
    }
  }
}

// out[g, c] = sum of the n rows of `part` from row g * n on.  32 columns per
// block, 16 threads per column, joined in a fixed order.
struct JoinP {
  const float* part[3];
  float* out[3];
  int n[3];        // rows joined into one
  int64_t first[3];  // first value of blockIdx.y of each
  int64_t D;
};
__global__ void __launch_bounds__(512) join_kernel(const JoinP p) {
  __shared__ float s[16][33];
  const int j = blockIdx.y >= p.first[2] ? 2 : blockIdx.y >= p.first[1] ? 1 : 0;
  const int64_t g = blockIdx.y - p.first[j];
  const int64_t c = int64_t(blockIdx.x) * 32 + threadIdx.x;
  float v = 0.0f;
  if (c < p.D) {
    const float* q = p.part[j] + g * p.n[j] * p.D + c;
    for (int i = threadIdx.y; i < p.n[j]; i += 16) v += q[int64_t(i) * p.D];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0 || c >= p.D) return;
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) v += s[i][threadIdx.x];
  p.out[j][g * p.D + c] = v;
}

// The backward's split, a function of the shape alone (for GB300's 152 SMs).
struct NormBwdPlan {
  int V, threads, grid;
  int64_t pieces, items;
};
NormBwdPlan norm_bwd_plan(int64_t M, int64_t D, int64_t gates) {
  NormBwdPlan q;
  const int64_t chunks = (D + 7) / 8;
  q.V = chunks <= 512 ? 1 : chunks <= 1024 ? 2 : 4;
  q.threads = int(((chunks + q.V - 1) / q.V + 31) / 32 * 32);
  const int per_sm = q.threads >= 512 ? 1 : 512 / q.threads > 8 ? 8 : 512 / q.threads;
  const int64_t blocks = 152 * per_sm;
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
  return q;
}

}  // namespace

cudaError_t launch_norm_fwd(const glu_block_norm_fwd_args& a, cudaStream_t s, const DevInfo& d) {
  NormFwdP p;
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
  return size_t(D) * 4 * (2 * size_t(q.grid) + (gates > 0 && q.pieces > 1 ? size_t(q.items) : 0));
}

template <typename XT>
static cudaError_t launch_bwd_t(const NormBwdP& p, const NormBwdPlan& q, cudaStream_t s) {
  switch (q.V) {
    case 1: return launch_kernel(norm_bwd_kernel<XT, 1>, q.grid, q.threads, 0, s, p);
    case 2: return launch_kernel(norm_bwd_kernel<XT, 2>, q.grid, q.threads, 0, s, p);
    default: return launch_kernel(norm_bwd_kernel<XT, 4>, q.grid, q.threads, 0, s, p);
  }
}

cudaError_t launch_norm_bwd(const glu_block_norm_bwd_args& a, cudaStream_t s) {
  const NormBwdPlan q = norm_bwd_plan(a.M, a.D, a.gates);
  NormBwdP p;
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
  p.part_post = p.part_pre + int64_t(q.grid) * a.D;
  p.part_gate = q.pieces > 1 ? p.part_post + int64_t(q.grid) * a.D : a.dgate;
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
  cudaError_t e = a.x_fmt == GLU_FMT_FP32 ? launch_bwd_t<float>(p, q, s) : launch_bwd_t<uint16_t>(p, q, s);
  if (e != cudaSuccess) return e;
  JoinP j;
  int64_t rows = 0;
  j.part[0] = p.part_pre, j.out[0] = a.dw_pre, j.n[0] = q.grid, j.first[0] = 0;
  rows += a.dw_pre ? 1 : 0;
  j.part[1] = p.part_post, j.out[1] = a.dw_post, j.n[1] = q.grid, j.first[1] = rows;
  rows += a.dw_post ? 1 : 0;
  j.part[2] = p.part_gate, j.out[2] = a.dgate, j.n[2] = int(q.pieces), j.first[2] = rows;
  rows += a.dgate && q.pieces > 1 ? a.gates : 0;
  j.D = a.D;
  if (rows == 0) return cudaSuccess;
  return launch_kernel(join_kernel, dim3(unsigned((a.D + 31) / 32), unsigned(rows)), dim3(32, 16), 0, s, j);
}

}  // namespace gq
