/*
 * glu_block8 — a transformer block's products and kept activations in 8-bit
 * floating point with a scale for each block of 128, for NVIDIA GB300
 * (sm_103a).  C ABI, next to glu_block.h, whose rules and status codes it
 * shares.
 *
 *   quantisers    matrices as E4M3 codes with fp32 scales;
 *   linear8       products of such operands, dense or by expert, with both
 *                 gradients;
 *   glu8          the gated activation that keeps gate and up in 8 bits, and
 *                 its backward from those.
 *
 * Format.  A block of 128 values v (fewer at the end of a dimension, as if
 * zeros followed) has a = max(max |v|, 2^-100), the scale s = a / 448 (fp32)
 * and the codes q = v * 448 / a rounded to E4M3 (to nearest, ties to even); it
 * stands for q * s.  Codes of bf16 values, and of products of two (glu8's h of ReLU
 * and the identity), are those of the exact quotient.  Others come from fp32
 * arithmetic: theirs are those of values within its error, to which the quotient adds
 * 2^-23 (relative).  That error is a few 2^-24 of a value, |t| 2^-21 where the
 * activation decays as e^-|t|, and relative to its terms where those cancel (dGate
 * next to a zero of act').  Quotients of codes, which have few bits, are often
 * midpoints between two codes, and may then get either.  A NaN or an infinity makes the
 * block's scale and codes NaN.  Three ways of cutting a matrix into blocks:
 *   rows     x [M, K]: 1 x 128.  q [M, K], s [ceil(K / 128), M].
 *   columns  x [M, K]: 128 x 1, for sums over the rows.  q [128 C, K], s
 *            [C, K]; dense, C = ceil(M / 128) and rows past M are zeros.  By
 *            expert, C = M / 128 (rounded down) + E: the rows of expert e
 *            begin at block offsets[e] / 128 + e, zeros follow its last one to
 *            the end of its last block, and blocks of no expert are zeros.
 *   weights  w [N, K], or a stack of E: 128 x 128.  q as w, s [ceil(N / 128),
 *            ceil(K / 128)], or a stack of E.
 *
 * Code matrices have a row stride (ld, in bytes) that is a multiple of 16, their
 * base 16-byte aligned; scales and offsets are contiguous, their base 4-byte
 * aligned (one matrix of a stack's serves).  offsets [E + 1]: device int32, from 0,
 * not falling, up to M; others are bounded (results are then undefined, no
 * access leaves the operands).  1 <= E <= 1024 by expert, E = 0 and offsets
 * NULL dense.  Outputs are fully overwritten up to the matrices' widths.
 */
#ifndef GLU_BLOCK8_H
#define GLU_BLOCK8_H

#include "glu_quant.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GLU_BLOCK8_ABI_VERSION 1

/* ---- quantisers --------------------------------------------------------
 * From x (bf16 [M, K]) the row form (q, s), the column form (qc, sc), or both
 * in one pass; or, x NULL, the column form of what the row form xq, xs stands
 * for.  E, offsets: experts of the column form (E = 0 without one). */
typedef struct glu_block8_quant_args {
  int64_t M, K;
  int64_t ld_x, ld_xq, ld_q, ld_qc;
  const void* x;
  const void* xq;
  const float* xs;
  const int32_t* offsets;
  void* q;
  float* s;
  void* qc;
  float* sc;
  int32_t E;
  int32_t reserved; /* 0 */
} glu_block8_quant_args;

/* w bf16 [N, K], or a stack of E (stride_w, stride_q between matrices). */
typedef struct glu_block8_quant_weight_args {
  int64_t N, K;
  int64_t ld_w, stride_w, ld_q, stride_q;
  const void* w;
  void* q;
  float* s;
  int32_t E;
  int32_t reserved; /* 0 */
} glu_block8_quant_weight_args;

GLU_API int glu_block8_quant(const glu_block8_quant_args* args, void* stream);
GLU_API int glu_block8_quant_weight(const glu_block8_quant_weight_args* args, void* stream);

/* ---- linear8 -----------------------------------------------------------
 * y = x W^T (grad 0: x [M, K] in row form, y bf16 [M, N]) or y = x W (grad 1,
 * the gradient of the input: x [M, N], y [M, K]), W [N, K] as weights.  The
 * tensor cores sum each block's 128 products; the blocks' sums are scaled, by the
 * fp32 product of the two scales, and added in fp32, in an order that depends on the
 * shapes only (a product of scales below 2^-126 loses bits, which is 2^-125 of a
 * result at most per block, and one above 2^128 is infinite).  By expert rows
 * offsets[e] .. offsets[e + 1] - 1 take W[e], rows from offsets[E] on give 0.
 * N, K <= 2^23.  The workspace (16-byte aligned; NULL where the query says 0)
 * joins the parts of sums that are split when there are few rows. */
typedef struct glu_block8_linear_args {
  int64_t M, N, K;
  int64_t ld_x, ld_w, stride_w, ld_y;
  const void* xq;
  const float* xs;
  const void* wq;
  const float* ws;
  const int32_t* offsets;
  void* y;
  void* workspace;
  size_t workspace_bytes;
  int32_t E;
  int32_t grad;
} glu_block8_linear_args;

/* dw = dy^T x ([N, K], or by expert [E, N, K]; bf16 or fp32, dw_fmt), dy [.., N]
 * and x [.., K] in column form of C blocks, with the same experts.  Experts
 * without rows get 0.  The workspace (16-byte aligned; NULL where the query says
 * 0) joins the parts of sums that are split where N and K are small. */
typedef struct glu_block8_linear_dw_args {
  int64_t C, N, K;
  int64_t ld_dy, ld_x, ld_dw, stride_dw;
  const void* dyq;
  const float* dys;
  const void* xq;
  const float* xs;
  const int32_t* offsets;
  void* dw;
  void* workspace;
  size_t workspace_bytes;
  int32_t E;
  int32_t dw_fmt; /* GLU_FMT_BF16 or GLU_FMT_FP32 */
} glu_block8_linear_dw_args;

GLU_API int glu_block8_linear(const glu_block8_linear_args* args, void* stream);
GLU_API int glu_block8_linear_workspace(const glu_block8_linear_args* args, size_t* bytes);
GLU_API int glu_block8_linear_dw(const glu_block8_linear_dw_args* args, void* stream);
GLU_API int glu_block8_linear_dw_workspace(const glu_block8_linear_dw_args* args, size_t* bytes);

/* ---- glu8 --------------------------------------------------------------
 * h = act(gate) .* up from gate, up bf16 [M, H], as bf16 (h) or in row form
 * (hq, hs; from the unrounded values), exactly one of them; gate and up kept
 * in row form (gq, gs, uq, us).  act: an enum glu_act without
 * GLU_ACT_BF16_STEPS. */
typedef struct glu_block8_glu_args {
  int64_t M, H;
  int64_t ld_gate, ld_up, ld_h, ld_hq, ld_gq, ld_uq;
  const void* gate;
  const void* up;
  void* h;
  void* hq;
  float* hs;
  void* gq;
  float* gs;
  void* uq;
  float* us;
  int32_t act;
  int32_t reserved; /* 0 */
} glu_block8_glu_args;

/* Backward, gate and up being what their row forms stand for:
 *   d = [dh .* up .* act'(gate) | dh .* act(gate)]  ([M, 2 H]),  h = act(gate) .* up
 * as bf16 (d; h or NULL), or quantised, without a rounding to bf16 between:
 * d in row form (dq, ds) and in column form (dqc, dsc), h in column form (hqc,
 * hsc, or both NULL).  The latter wants H a multiple of 128; offsets and E are
 * those of the column forms.  Far out act' of SiLU and the GELUs is 0 and 1;
 * ReLU's is 0 up to 0. */
typedef struct glu_block8_glu_bwd_args {
  int64_t M, H;
  int64_t ld_gq, ld_uq, ld_dh, ld_d, ld_h, ld_dq, ld_dqc, ld_hqc;
  const void* gq;
  const float* gs;
  const void* uq;
  const float* us;
  const void* dh;
  const int32_t* offsets;
  void* d;
  void* h;
  void* dq;
  float* ds;
  void* dqc;
  float* dsc;
  void* hqc;
  float* hsc;
  int32_t act;
  int32_t E;
} glu_block8_glu_bwd_args;

GLU_API int glu_block8_glu(const glu_block8_glu_args* args, void* stream);
GLU_API int glu_block8_glu_bwd(const glu_block8_glu_bwd_args* args, void* stream);

GLU_API int glu_block8_abi_version(void);

/* Bounded waits of these kernels that gave up show in glu_block_device_errors. */

#ifdef __cplusplus
}
#endif
#endif /* GLU_BLOCK8_H */
