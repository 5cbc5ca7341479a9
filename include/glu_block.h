/*
 * glu_block — the operators around a gated activation in a transformer
 * block, for NVIDIA GB300 (sm_103a).  C ABI, next to glu_quant.h, whose
 * status codes, enums and rules it shares.
 *
 *   block norms   r = x + alpha * gate .* P(branch), y = N(r) and their
 *                 gradients (N, P: RMS norms with weights);
 *   routing       tokens sorted by expert and back, with the router's
 *                 weights, and the gradients;
 *   linear        y = act(x W^T + b) + residual, dense or with one W per
 *                 expert over sorted rows, and its gradients.
 *
 * Rules (as in glu_quant.h): every pointer is a DEVICE pointer owned by the
 * caller; nothing is allocated, freed or synchronised; launches go to
 * `stream` only and can be captured in a CUDA graph; every argument is
 * checked before the first launch, and only GLU_ELAUNCH may leave outputs
 * partly written.  Outputs are fully overwritten and must not alias inputs.
 * Matrices are row-major with a row stride (ld, in elements) that is a
 * multiple of 8, their base 16-byte aligned (GLU_EALIGN otherwise); the
 * widths themselves are free.  Every other pointer is 16-byte aligned too, and
 * what it points to contiguous.  A call with several launches orders them on
 * the stream; workspaces may be reused by the next call on that stream.
 * Indices that a call reads from device memory (offsets, slot, src) are
 * bounded in the kernels: one out of range counts as dropped.  Sums (norm
 * statistics, products, gradients of shared operands) are fp32, taken in an
 * order that depends on the shapes only, so that a call gives the same bits
 * every time.  What stands between the end of a row and the next row (ld above
 * the width) is never written and never counts; glu_block_combine and
 * glu_block_combine_bwd read up to seven elements of it behind rows_in's rows,
 * so nothing else may write there while they run.
 */
#ifndef GLU_BLOCK_H
#define GLU_BLOCK_H

#include "glu_quant.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GLU_BLOCK_ABI_VERSION 1

/* ---- block norms -------------------------------------------------------
 * Forward, for every row m of M (all in fp32, rounded once at the stores):
 *   P = branch_m                                          (w_post NULL)
 *     = branch_m * rstd_post[m] .* (w_post + w_offset)     (w_post given)
 *   r_m = x_m + alpha * gate_g .* P           (branch given; else r_m = x_m)
 *   y_m = r_m * rstd_pre[m] .* (w_pre + w_offset)         (w_pre given)
 *   rstd(v) = 1 / sqrt(sum(v^2) / D + eps)
 * gate [gates, D]: row m takes row m / (M / gates) (gates divides M; 1: one
 * row for all, M: one per row; gate NULL means 1, gates 0).  y is formed
 * from r before r is rounded.  x and r are bf16 or fp32 (x_fmt), branch, gate
 * and y bf16, the weights bf16 or fp32 (w_fmt), the rstd fp32.
 * Outputs, NULL exactly when not produced: r (branch given), y and rstd_pre
 * (w_pre given), rstd_post (w_post given).  At least one of branch and w_pre
 * is given; w_post and gate need branch.  1 <= D <= 32768 (the row stays in
 * registers). */
typedef struct glu_block_norm_fwd_args {
  int32_t x_fmt; /* GLU_FMT_BF16 or GLU_FMT_FP32: x, r */
  int32_t w_fmt; /* GLU_FMT_BF16 or GLU_FMT_FP32: w_pre, w_post */
  float alpha, w_offset, eps;
  int32_t reserved; /* 0 */
  int64_t M, D, gates;
  int64_t ld_x, ld_branch, ld_gate, ld_r, ld_y;
  const void* x;
  const void* branch;
  const void* gate;
  const void* w_pre;
  const void* w_post;
  void* r;
  void* y;
  float* rstd_pre;
  float* rstd_post;
} glu_block_norm_fwd_args;

/* Backward: from dy (gradient of y; given exactly when w_pre is) and dr
 * (gradient of r from elsewhere; NULL: none), with r, branch, gate, the
 * weights and the rstd of the forward:
 *   dR = dr + rstd_pre * (u - n * sum(u n) / D), u = dy .* (w_pre + w_offset),
 *        n = r * rstd_pre                        (w_pre NULL: dR = dr)
 *   dx = dR;  dw_pre = sum_m dy .* n
 *   dgate_g = alpha * sum over the rows of g of dR .* P
 *   d = alpha * gate .* dR;  dbranch = d                   (w_post NULL)
 *   dbranch = rstd_post * (u' - n' * sum(u' n') / D), u' = d .* (w_post +
 *        w_offset), n' = branch * rstd_post;  dw_post = sum_m d .* n'
 * r, dr and dx have x_fmt; dbranch is bf16; dw_pre, dw_post [D] and dgate
 * [gates, D] (contiguous) are fp32.  NULL exactly when not produced: dw_pre
 * (w_pre), dbranch (branch), dw_post (w_post), dgate (gate); r may be NULL
 * when w_pre is.  1 <= D <= 16384.  The workspace (16-byte aligned) holds
 * the partial sums; its size is glu_block_norm_bwd_workspace's. */
typedef struct glu_block_norm_bwd_args {
  int32_t x_fmt, w_fmt;
  float alpha, w_offset;
  int64_t M, D, gates;
  int64_t ld_r, ld_branch, ld_gate, ld_dy, ld_dr, ld_dx, ld_dbranch;
  const void* r;
  const void* branch;
  const void* gate;
  const void* w_pre;
  const void* w_post;
  const float* rstd_pre;
  const float* rstd_post;
  const void* dy;
  const void* dr;
  void* dx;
  void* dbranch;
  float* dw_pre;
  float* dw_post;
  float* dgate;
  void* workspace;
  size_t workspace_bytes;
} glu_block_norm_bwd_args;

GLU_API int glu_block_norm_fwd(const glu_block_norm_fwd_args* args, void* stream);
GLU_API int glu_block_norm_bwd(const glu_block_norm_bwd_args* args, void* stream);
/* Bytes of workspace that a backward of M rows of width D, with `gates` gate
 * rows, needs on any device (an upper bound; touches no device). */
GLU_API int glu_block_norm_bwd_workspace(int64_t M, int64_t D, int64_t gates, size_t* bytes);

/* ---- expert routing ----------------------------------------------------
 * ids [T, K] (contiguous int32 or int64): the experts of each token; a value
 * outside [0, E) is an assignment that was dropped.  glu_block_route sorts
 * the assignments j = t * K + k by expert, keeping their order inside one:
 *   offsets [E + 1]: expert e has the places offsets[e] .. offsets[e + 1] - 1
 *   slot [T, K]:     the place of (t, k), -1 where it was dropped
 *   src [T * K]:     the j at each place, -1 from offsets[E] on
 * (all int32).  1 <= T * K < 2^31, 1 <= E <= 1024.  The workspace (16-byte
 * aligned; NULL where the query says 0) has glu_block_route_workspace's
 * bytes. */
typedef struct glu_block_route_args {
  int32_t id_bytes; /* 4 or 8 */
  int32_t E;
  int64_t T, K;
  const void* ids;
  int32_t* slot;
  int32_t* src;
  int32_t* offsets;
  void* workspace;
  size_t workspace_bytes;
} glu_block_route_args;

GLU_API int glu_block_route(const glu_block_route_args* args, void* stream);
GLU_API int glu_block_route_workspace(int64_t T, int64_t K, int32_t E, size_t* bytes);

/* Rows of width D (bf16) by the places of a route, R = T * K of them:
 *   dispatch:     rows_out[p] = x[src[p] / K]; 0 where src[p] < 0
 *   combine:      out[t] = residual[t] + sum_k w[t, k] * rows_in[slot[t, k]]
 *                 (residual NULL: none; w NULL: 1, which makes it the
 *                 gradient of dispatch; slots < 0 add nothing)
 *   combine_bwd:  drows[p] = w[src[p]] * dout[src[p] / K], 0 where src[p] < 0;
 *                 dw[t, k] = <rows_in[slot[t, k]], dout[t]>, 0 where slot < 0
 * w and dw are contiguous fp32 [T, K].  slot and src are a route's: every
 * slot below R, every src below T * K, each the inverse of the other. */
typedef struct glu_block_rows_args {
  int64_t T, K, D;
  int64_t ld_tokens;   /* x, out, dout */
  int64_t ld_rows;     /* rows_in */
  int64_t ld_rows_out; /* rows_out, drows */
  int64_t ld_residual;
  const int32_t* slot;
  const int32_t* src;
  const float* w;
  const void* tokens_in;   /* dispatch: x; combine_bwd: dout */
  const void* rows_in;     /* combine, combine_bwd */
  const void* residual;    /* combine */
  void* tokens_out;        /* combine */
  void* rows_out;          /* dispatch; combine_bwd: drows */
  float* dw;               /* combine_bwd */
} glu_block_rows_args;

GLU_API int glu_block_dispatch(const glu_block_rows_args* args, void* stream);
GLU_API int glu_block_combine(const glu_block_rows_args* args, void* stream);
GLU_API int glu_block_combine_bwd(const glu_block_rows_args* args, void* stream);

/* ---- linear ------------------------------------------------------------
 * z = x W^T + bias, y = act(z) + residual: x [M, K], W [N, K], residual and y
 * [M, N] bf16, products summed in fp32 on the tensor cores; z (bf16) is
 * stored where its pointer is given, y is formed from z before it is rounded.
 * act: an enum glu_act without GLU_ACT_BF16_STEPS (GLU_ACT_IDENTITY: none).
 * By expert: E > 0, W [E, N, K] (stride_w elements between experts), bias
 * [E, N], and offsets [E + 1] (device int32, from 0, not falling): rows
 * offsets[e] .. offsets[e + 1] - 1 of x take W[e]; rows from offsets[E] on
 * give y = z = 0.  Dense: E = 0, offsets NULL.  E <= 1024, N and K <= 2^23.
 * The workspace (16-byte aligned; NULL where the query says 0 bytes) joins
 * the parts of long sums that are split when there are few rows. */
typedef struct glu_block_linear_fwd_args {
  int32_t act;
  int32_t b_fmt; /* GLU_FMT_BF16 or GLU_FMT_FP32: bias */
  int32_t E;
  int32_t reserved; /* 0 */
  int64_t M, N, K;
  int64_t ld_x, ld_w, stride_w, ld_residual, ld_y, ld_z;
  const void* x;
  const void* w;
  const void* bias;     /* or NULL */
  const void* residual; /* or NULL */
  const int32_t* offsets;
  void* y;
  void* z; /* or NULL */
  void* workspace;
  size_t workspace_bytes;
} glu_block_linear_fwd_args;

/* Backward: dz = dy .* act'(z) (act = GLU_ACT_IDENTITY: dz = dy, z NULL;
 * act' of SiLU and the GELUs is 0 and 1 at -inf and +inf, their limits),
 *   dx = dz W (bf16 [M, K]), dw = dz^T x (bf16, W's shape), db = sum over the
 *   rows of dz (fp32 [N], by expert [E, N]); each is skipped where its
 *   pointer is NULL.  dz is rounded to bf16 for the products (the tensor
 *   cores take bf16 operands), not for db.  The gradient of residual is dy.
 * Experts without rows get dw = db = 0; rows from offsets[E] on dx = 0. */
typedef struct glu_block_linear_bwd_args {
  int32_t act;
  int32_t E;
  int64_t M, N, K;
  int64_t ld_dy, ld_z, ld_x, ld_w, stride_w, ld_dx, ld_dw, stride_dw;
  const void* dy;
  const void* z;
  const void* x; /* needed for dw */
  const void* w; /* needed for dx */
  const int32_t* offsets;
  void* dx;
  void* dw;
  float* db;
  void* workspace;
  size_t workspace_bytes;
} glu_block_linear_bwd_args;

GLU_API int glu_block_linear_fwd(const glu_block_linear_fwd_args* args, void* stream);
GLU_API int glu_block_linear_bwd(const glu_block_linear_bwd_args* args, void* stream);
/* Bytes of workspace for these arguments (pointers are looked at only for
 * being NULL; the workspace fields are not). */
GLU_API int glu_block_linear_fwd_workspace(const glu_block_linear_fwd_args* args, size_t* bytes);
GLU_API int glu_block_linear_bwd_workspace(const glu_block_linear_bwd_args* args, size_t* bytes);

/* As glu_quant_device_errors, for the kernels of this header and of glu_block8.h. */
GLU_API int glu_block_device_errors(uint32_t* bits, int clear);
GLU_API int glu_block_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* GLU_BLOCK_H */
