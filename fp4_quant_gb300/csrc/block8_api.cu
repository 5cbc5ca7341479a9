// C ABI of the operators in 8 bits (include/glu_block8.h): the checks of every
// argument, before anything is launched, and the launches.
#include <climits>

#include "block8.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A given [rows, cols] matrix of elements of `size` bytes: row stride and the
// bytes it spans (ESHAPE), rows on 16 bytes (EALIGN).  An absent one is fine.
struct Check {
  int status = GLU_OK;
  void fail(int st) {
    if (status == GLU_OK) status = st;
  }
  void matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int size) {
    if (p == nullptr) return;
    int64_t t;
    if (ld < cols || __builtin_mul_overflow(rows, ld, &t) || __builtin_mul_overflow(t, int64_t(8), &t)) fail(GLU_ESHAPE);
    else if (ld * size % 16 != 0 || !aligned16(p)) fail(GLU_EALIGN);
  }
  // E of them, `stride` elements apart (E = 0: one)
  void stack(const void* p, int32_t E, int64_t rows, int64_t cols, int64_t ld, int64_t stride, int size) {
    matrix(p, rows, cols, ld, size);
    if (p == nullptr || E == 0 || status != GLU_OK) return;
    int64_t t;
    if (stride < rows * ld || __builtin_mul_overflow(stride, int64_t(E), &t) || __builtin_mul_overflow(t, int64_t(8), &t) ||
        stride >= (int64_t(1) << 38))
      fail(GLU_ESHAPE);
    else if (stride * size % 16 != 0) fail(GLU_EALIGN);
  }
  // scales and offsets are read by the word: parts of a stack's serve too
  void words(const void* p) {
    if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) fail(GLU_EALIGN);
  }
};

int launched(cudaError_t e) {
  if (e == cudaSuccess) return GLU_OK;
  cudaGetLastError();  // the launch error is reported through the status
  return GLU_ELAUNCH;
}

// 32-bit rows, columns and TMA coordinates, and grids of tiles below 2^30.
constexpr int64_t kMostRows = INT32_MAX - 1024, kWidest = int64_t(1) << 23;
int check_size(int64_t M, int64_t K, int32_t E) {
  if (M <= 0 || K <= 0 || E < 0) return GLU_EINVAL;
  if (M > kMostRows || K > kWidest || E > gq::kMaxExperts) return GLU_ESHAPE;
  const int64_t rows = (M / gq::kBlock8 + 2 + E) * gq::kBlock8;  // of a column form, and one tile more
  return rows > kMostRows || rows / 64 * gq::blocks8(K) > (int64_t(1) << 30) ? GLU_ESHAPE : GLU_OK;
}
int check_weight_size(int64_t N, int64_t K, int32_t E) {
  if (N <= 0 || K <= 0 || E < 0) return GLU_EINVAL;
  if (N > kWidest || K > kWidest || E > gq::kMaxExperts) return GLU_ESHAPE;
  return gq::blocks8(N) * gq::blocks8(K) * (E > 0 ? E : 1) > (int64_t(1) << 30) ? GLU_ESHAPE : GLU_OK;
}
bool act_ok(int32_t act) { return act >= GLU_ACT_SILU && act <= GLU_ACT_GELU_ERF; }
bool both_or_none(const void* a, const void* b) { return (a != nullptr) == (b != nullptr); }

int check_quant(const glu_block8_quant_args* a) {
  if (a == nullptr || a->reserved != 0) return GLU_EINVAL;
  const int st = check_size(a->M, a->K, a->E);
  if (st != GLU_OK) return st;
  const bool kept = a->xq != nullptr;
  if ((a->x != nullptr) == kept || !both_or_none(a->xq, a->xs) || !both_or_none(a->q, a->s) || !both_or_none(a->qc, a->sc)) return GLU_EINVAL;
  if ((!a->q && !a->qc) || (kept && a->q) || (a->offsets != nullptr) != (a->E > 0) || (a->E > 0 && !a->qc)) return GLU_EINVAL;
  Check c;
  c.matrix(a->x, a->M, a->K, a->ld_x, 2);
  c.matrix(a->xq, a->M, a->K, a->ld_xq, 1);
  c.matrix(a->q, a->M, a->K, a->ld_q, 1);
  c.matrix(a->qc, gq::col_blocks8(a->M, a->E) * gq::kBlock8, a->K, a->ld_qc, 1);
  for (const void* p : {static_cast<const void*>(a->xs), static_cast<const void*>(a->offsets), static_cast<const void*>(a->s),
                        static_cast<const void*>(a->sc)})
    c.words(p);
  return c.status;
}

int check_quant_weight(const glu_block8_quant_weight_args* a) {
  if (a == nullptr || a->reserved != 0) return GLU_EINVAL;
  const int st = check_weight_size(a->N, a->K, a->E);
  if (st != GLU_OK) return st;
  if (!a->w || !a->q || !a->s) return GLU_EINVAL;
  Check c;
  c.stack(a->w, a->E, a->N, a->K, a->ld_w, a->stride_w, 2);
  c.stack(a->q, a->E, a->N, a->K, a->ld_q, a->stride_q, 1);
  c.words(a->s);
  return c.status;
}

int check_linear(const glu_block8_linear_args* a, bool query) {
  if (a == nullptr || (a->grad != 0 && a->grad != 1)) return GLU_EINVAL;
  int st = check_size(a->M, a->N > a->K ? a->N : a->K, a->E);
  if (st == GLU_OK) st = check_weight_size(a->N, a->K, a->E);
  if (st != GLU_OK) return st;
  if (query) return GLU_OK;
  if (!a->xq || !a->xs || !a->wq || !a->ws || !a->y || (a->offsets != nullptr) != (a->E > 0)) return GLU_EINVAL;
  const size_t need = gq::linear8_workspace(*a);
  if (need > 0 && (a->workspace == nullptr || a->workspace_bytes < need)) return GLU_EINVAL;
  const bool grad = a->grad != 0;
  Check c;
  c.matrix(a->xq, a->M, grad ? a->N : a->K, a->ld_x, 1);
  c.stack(a->wq, a->E, a->N, a->K, a->ld_w, a->stride_w, 1);
  c.matrix(a->y, a->M, grad ? a->K : a->N, a->ld_y, 2);
  for (const void* p : {static_cast<const void*>(a->xs), static_cast<const void*>(a->ws), static_cast<const void*>(a->offsets)})
    c.words(p);
  if (need > 0 && !aligned16(a->workspace)) c.fail(GLU_EALIGN);
  return c.status;
}

int check_linear_dw(const glu_block8_linear_dw_args* a, bool query) {
  if (a == nullptr || (a->dw_fmt != GLU_FMT_BF16 && a->dw_fmt != GLU_FMT_FP32) || a->C <= 0) return GLU_EINVAL;
  int st = check_weight_size(a->N, a->K, a->E);
  if (st != GLU_OK) return st;
  if (a->C > kMostRows / gq::kBlock8) return GLU_ESHAPE;
  if (query) return a->C < a->E ? GLU_EINVAL : GLU_OK;
  if (!a->dyq || !a->dys || !a->xq || !a->xs || !a->dw || (a->offsets != nullptr) != (a->E > 0) || a->C < a->E) return GLU_EINVAL;
  const size_t need = gq::linear8_dw_workspace(*a);
  if (need > 0 && (a->workspace == nullptr || a->workspace_bytes < need)) return GLU_EINVAL;
  const int64_t rows = a->C * gq::kBlock8;
  const int size = a->dw_fmt == GLU_FMT_FP32 ? 4 : 2;
  Check c;
  c.matrix(a->dyq, rows, a->N, a->ld_dy, 1);
  c.matrix(a->xq, rows, a->K, a->ld_x, 1);
  c.stack(a->dw, a->E, a->N, a->K, a->ld_dw, a->stride_dw, size);
  for (const void* p : {static_cast<const void*>(a->dys), static_cast<const void*>(a->xs), static_cast<const void*>(a->offsets)}) c.words(p);
  if (need > 0 && !aligned16(a->workspace)) c.fail(GLU_EALIGN);
  return c.status;
}

int check_glu(const glu_block8_glu_args* a) {
  if (a == nullptr || !act_ok(a->act) || a->reserved != 0) return GLU_EINVAL;
  const int st = check_size(a->M, a->H, 0);
  if (st != GLU_OK) return st;
  if (!a->gate || !a->up || !a->gq || !a->gs || !a->uq || !a->us || (a->h != nullptr) == (a->hq != nullptr) || !both_or_none(a->hq, a->hs))
    return GLU_EINVAL;
  Check c;
  c.matrix(a->gate, a->M, a->H, a->ld_gate, 2);
  c.matrix(a->up, a->M, a->H, a->ld_up, 2);
  c.matrix(a->h, a->M, a->H, a->ld_h, 2);
  c.matrix(a->hq, a->M, a->H, a->ld_hq, 1);
  c.matrix(a->gq, a->M, a->H, a->ld_gq, 1);
  c.matrix(a->uq, a->M, a->H, a->ld_uq, 1);
  for (const void* p : {static_cast<const void*>(a->hs), static_cast<const void*>(a->gs), static_cast<const void*>(a->us)}) c.words(p);
  return c.status;
}

int check_glu_bwd(const glu_block8_glu_bwd_args* a) {
  if (a == nullptr || !act_ok(a->act) || a->M <= 0 || a->H <= 0 || a->E < 0) return GLU_EINVAL;
  if (a->H > kWidest / 2) return GLU_ESHAPE;
  const int st = check_size(a->M, 2 * a->H, a->E);
  if (st != GLU_OK) return st;
  if (!a->gq || !a->gs || !a->uq || !a->us || !a->dh || (a->offsets != nullptr) != (a->E > 0)) return GLU_EINVAL;
  const bool plain = a->d != nullptr;
  if ((a->dq != nullptr) == plain || (a->ds != nullptr) == plain || (a->dqc != nullptr) == plain || (a->dsc != nullptr) == plain) return GLU_EINVAL;
  if (!both_or_none(a->hqc, a->hsc) || (plain && (a->hqc || a->E > 0)) || (!plain && a->h)) return GLU_EINVAL;
  if (!plain && a->H % gq::kBlock8 != 0) return GLU_ESHAPE;
  const int64_t cols = gq::col_blocks8(a->M, a->E) * gq::kBlock8;
  Check c;
  c.matrix(a->gq, a->M, a->H, a->ld_gq, 1);
  c.matrix(a->uq, a->M, a->H, a->ld_uq, 1);
  c.matrix(a->dh, a->M, a->H, a->ld_dh, 2);
  c.matrix(a->d, a->M, 2 * a->H, a->ld_d, 2);
  c.matrix(a->h, a->M, a->H, a->ld_h, 2);
  c.matrix(a->dq, a->M, 2 * a->H, a->ld_dq, 1);
  c.matrix(a->dqc, cols, 2 * a->H, a->ld_dqc, 1);
  c.matrix(a->hqc, cols, a->H, a->ld_hqc, 1);
  for (const void* p : {static_cast<const void*>(a->gs), static_cast<const void*>(a->us), static_cast<const void*>(a->offsets),
                        static_cast<const void*>(a->ds), static_cast<const void*>(a->dsc), static_cast<const void*>(a->hsc)})
    c.words(p);
  return c.status;
}

}  // namespace

// Every entry point: its checks, the device, the launch.
#define GQ_ENTRY(check, launch)                             \
  const int st = (check);                                   \
  if (st != GLU_OK) return st;                              \
  gq::DevInfo d;                                            \
  const int dev = gq::device_info(&d);                      \
  if (dev != GLU_OK) return dev;                            \
  const cudaStream_t s = static_cast<cudaStream_t>(stream); \
  return launched(launch)

extern "C" int glu_block8_quant(const glu_block8_quant_args* a, void* stream) { GQ_ENTRY(check_quant(a), gq::launch_quant8(*a, s, d)); }
extern "C" int glu_block8_quant_weight(const glu_block8_quant_weight_args* a, void* stream) {
  GQ_ENTRY(check_quant_weight(a), gq::launch_quant8_weight(*a, s));
}
extern "C" int glu_block8_linear(const glu_block8_linear_args* a, void* stream) {
  GQ_ENTRY(check_linear(a, false), gq::launch_linear8(*a, s, d));
}
extern "C" int glu_block8_linear_dw(const glu_block8_linear_dw_args* a, void* stream) {
  GQ_ENTRY(check_linear_dw(a, false), gq::launch_linear8_dw(*a, s, d));
}
extern "C" int glu_block8_glu(const glu_block8_glu_args* a, void* stream) { GQ_ENTRY(check_glu(a), gq::launch_glu8(*a, s)); }
extern "C" int glu_block8_glu_bwd(const glu_block8_glu_bwd_args* a, void* stream) {
  GQ_ENTRY(check_glu_bwd(a), gq::launch_glu8_bwd(*a, s, d));
}
extern "C" int glu_block8_linear_workspace(const glu_block8_linear_args* a, size_t* bytes) {
  if (bytes == nullptr) return GLU_EINVAL;
  const int st = check_linear(a, true);
  if (st == GLU_OK) *bytes = gq::linear8_workspace(*a);
  return st;
}
extern "C" int glu_block8_linear_dw_workspace(const glu_block8_linear_dw_args* a, size_t* bytes) {
  if (bytes == nullptr) return GLU_EINVAL;
  const int st = check_linear_dw(a, true);
  if (st == GLU_OK) *bytes = gq::linear8_dw_workspace(*a);
  return st;
}
extern "C" int glu_block8_abi_version(void) { return GLU_BLOCK8_ABI_VERSION; }
