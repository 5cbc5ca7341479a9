// C ABI of the block operators (include/glu_block.h): the checks of every
// argument, before anything is launched, and the launches.
#include <climits>

#include "block8.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool float_fmt(int32_t f) { return f == GLU_FMT_BF16 || f == GLU_FMT_FP32; }

// A given [rows, cols] matrix: row stride and the bytes it spans (ESHAPE),
// its alignment (EALIGN).  An absent one is fine.
struct Check {
  int status = GLU_OK;
  void fail(int st) {
    if (status == GLU_OK) status = st;
  }
  void matrix(const void* p, int64_t rows, int64_t cols, int64_t ld) {
    if (p == nullptr) return;
    int64_t t;
    if (ld < cols || __builtin_mul_overflow(rows, ld, &t) || __builtin_mul_overflow(t, int64_t(4), &t)) fail(GLU_ESHAPE);
    else if (ld % 8 != 0 || !aligned16(p)) fail(GLU_EALIGN);
  }
  void vec(const void* p) {
    if (p != nullptr && !aligned16(p)) fail(GLU_EALIGN);
  }
};

int launched(cudaError_t e) {
  if (e == cudaSuccess) return GLU_OK;
  cudaGetLastError();  // the launch error is reported through the status
  return GLU_ELAUNCH;
}

constexpr int64_t kMaxNormFwd = 32768, kMaxNormBwd = 16384;

int check_gates(int64_t M, int64_t gates, const void* gate) {
  if ((gate != nullptr) != (gates > 0) || gates < 0) return GLU_EINVAL;
  return gates > 0 && M % gates != 0 ? GLU_ESHAPE : GLU_OK;
}

int check_norm_fwd(const glu_block_norm_fwd_args* a) {
  if (a == nullptr || !float_fmt(a->x_fmt) || !float_fmt(a->w_fmt) || a->reserved != 0) return GLU_EINVAL;
  if (a->M <= 0 || a->D <= 0 || a->x == nullptr) return GLU_EINVAL;
  const bool br = a->branch != nullptr, pre = a->w_pre != nullptr, post = a->w_post != nullptr;
  if ((!br && !pre) || (post && !br) || (a->gate != nullptr && !br)) return GLU_EINVAL;
  if ((a->r != nullptr) != br || (a->y != nullptr) != pre || (a->rstd_pre != nullptr) != pre || (a->rstd_post != nullptr) != post)
    return GLU_EINVAL;
  const int st = check_gates(a->M, a->gates, a->gate);
  if (st != GLU_OK) return st;
  if (a->D > kMaxNormFwd) return GLU_ESHAPE;
  Check c;
  c.matrix(a->x, a->M, a->D, a->ld_x);
  c.matrix(a->branch, a->M, a->D, a->ld_branch);
  c.matrix(a->gate, a->gates, a->D, a->ld_gate);
  c.matrix(a->r, a->M, a->D, a->ld_r);
  c.matrix(a->y, a->M, a->D, a->ld_y);
  for (const void* p : {a->w_pre, a->w_post, static_cast<const void*>(a->rstd_pre), static_cast<const void*>(a->rstd_post)}) c.vec(p);
  return c.status;
}

int check_norm_bwd(const glu_block_norm_bwd_args* a) {
  if (a == nullptr || !float_fmt(a->x_fmt) || !float_fmt(a->w_fmt)) return GLU_EINVAL;
  if (a->M <= 0 || a->D <= 0 || a->dx == nullptr) return GLU_EINVAL;
  const bool br = a->branch != nullptr, pre = a->w_pre != nullptr, post = a->w_post != nullptr;
  if ((!br && !pre) || (post && !br) || (a->gate != nullptr && !br)) return GLU_EINVAL;
  if (pre && (a->r == nullptr || a->rstd_pre == nullptr)) return GLU_EINVAL;
  if (post && a->rstd_post == nullptr) return GLU_EINVAL;
  if ((a->dy != nullptr) != pre || (!pre && a->dr == nullptr)) return GLU_EINVAL;
  if ((a->dw_pre != nullptr) != pre || (a->dw_post != nullptr) != post || (a->dbranch != nullptr) != br ||
      (a->dgate != nullptr) != (a->gate != nullptr))
    return GLU_EINVAL;
  const int st = check_gates(a->M, a->gates, a->gate);
  if (st != GLU_OK) return st;
  if (a->D > kMaxNormBwd) return GLU_ESHAPE;
  if (a->workspace == nullptr || a->workspace_bytes < gq::norm_bwd_workspace(a->M, a->D, a->gates)) return GLU_EINVAL;
  Check c;
  c.matrix(a->r, a->M, a->D, a->ld_r);
  c.matrix(a->branch, a->M, a->D, a->ld_branch);
  c.matrix(a->gate, a->gates, a->D, a->ld_gate);
  c.matrix(a->dy, a->M, a->D, a->ld_dy);
  c.matrix(a->dr, a->M, a->D, a->ld_dr);
  c.matrix(a->dx, a->M, a->D, a->ld_dx);
  c.matrix(a->dbranch, a->M, a->D, a->ld_dbranch);
  for (const void* p : {a->w_pre, a->w_post, static_cast<const void*>(a->rstd_pre), static_cast<const void*>(a->rstd_post),
                        static_cast<const void*>(a->dw_pre), static_cast<const void*>(a->dw_post),
                        static_cast<const void*>(a->dgate), static_cast<const void*>(a->workspace)})
    c.vec(p);
  return c.status;
}

int check_route_size(int64_t T, int64_t K, int32_t E) {
  if (T <= 0 || K <= 0 || E <= 0) return GLU_EINVAL;
  int64_t n;
  return E > gq::kMaxExperts || __builtin_mul_overflow(T, K, &n) || n > INT32_MAX ? GLU_ESHAPE : GLU_OK;
}

int check_route(const glu_block_route_args* a) {
  if (a == nullptr || (a->id_bytes != 4 && a->id_bytes != 8)) return GLU_EINVAL;
  const int st = check_route_size(a->T, a->K, a->E);
  if (st != GLU_OK) return st;
  if (!a->ids || !a->slot || !a->src || !a->offsets) return GLU_EINVAL;
  const size_t need = gq::route_workspace(a->T, a->K, a->E);
  if (need > 0 && (a->workspace == nullptr || a->workspace_bytes < need)) return GLU_EINVAL;
  Check c;
  for (const void* p : {a->ids, static_cast<const void*>(a->slot), static_cast<const void*>(a->src),
                        static_cast<const void*>(a->offsets), static_cast<const void*>(a->workspace)})
    c.vec(p);
  return c.status;
}

enum RowsOp { kDispatch, kCombine, kCombineBwd };

int check_rows(const glu_block_rows_args* a, RowsOp op) {
  if (a == nullptr || a->T <= 0 || a->K <= 0 || a->D <= 0 || a->slot == nullptr) return GLU_EINVAL;
  const bool in = op != kCombine, rows_in = op != kDispatch, out = op == kCombine;
  if ((a->tokens_in != nullptr) != in || (a->rows_in != nullptr) != rows_in || (a->tokens_out != nullptr) != out ||
      (a->rows_out != nullptr) != !out || (a->dw != nullptr) != (op == kCombineBwd) || (a->residual != nullptr && !out) ||
      (a->w == nullptr && op == kCombineBwd) || (a->w != nullptr && op == kDispatch) || (a->src != nullptr) != !out)
    return GLU_EINVAL;
  int64_t R;
  if (__builtin_mul_overflow(a->T, a->K, &R) || R > INT32_MAX || a->D > INT32_MAX - 1024) return GLU_ESHAPE;
  Check c;
  c.matrix(out ? a->tokens_out : a->tokens_in, a->T, a->D, a->ld_tokens);
  c.matrix(a->rows_in, R, a->D, a->ld_rows);
  c.matrix(a->rows_out, R, a->D, a->ld_rows_out);
  c.matrix(a->residual, a->T, a->D, a->ld_residual);
  for (const void* p : {static_cast<const void*>(a->slot), static_cast<const void*>(a->src), static_cast<const void*>(a->w),
                        static_cast<const void*>(a->dw)})
    c.vec(p);
  return c.status;
}

// Sizes of a linear layer: 32-bit TMA coordinates, grids over N and K, and tiles
// counted in 31 bits.
int check_linear_size(int64_t M, int64_t N, int64_t K, int32_t E) {
  if (M <= 0 || N <= 0 || K <= 0 || E < 0) return GLU_EINVAL;
  constexpr int64_t kMost = INT32_MAX - 1024;
  constexpr int64_t kWidest = int64_t(1) << 23;
  if (M > kMost || N > kWidest || K > kWidest || E > gq::kMaxExperts) return GLU_ESHAPE;
  const int64_t m = M / 128 + 1 + E, n = N / 128 + 1, k = K / 128 + 1, most = int64_t(1) << 30;
  return m * n > most || m * k > most || n * k * (E > 0 ? E : 1) > most ? GLU_ESHAPE : GLU_OK;
}

void weights(Check& c, const void* w, int32_t E, int64_t N, int64_t K, int64_t ld, int64_t stride) {
  c.matrix(w, N, K, ld);
  if (w == nullptr || E == 0) return;
  int64_t t;
  if (stride < N * ld || __builtin_mul_overflow(stride, int64_t(E), &t) || __builtin_mul_overflow(t, int64_t(2), &t) ||
      stride >= (int64_t(1) << 38))
    c.fail(GLU_ESHAPE);
  else if (stride % 8 != 0) c.fail(GLU_EALIGN);
}

int check_linear_fwd(const glu_block_linear_fwd_args* a, bool query) {
  if (a == nullptr || a->act < GLU_ACT_SILU || a->act > GLU_ACT_GELU_ERF || !float_fmt(a->b_fmt) || a->reserved != 0) return GLU_EINVAL;
  const int st = check_linear_size(a->M, a->N, a->K, a->E);
  if (st != GLU_OK) return st;
  if (query) return GLU_OK;
  if (!a->x || !a->w || !a->y || (a->offsets != nullptr) != (a->E > 0)) return GLU_EINVAL;
  const size_t need = gq::linear_fwd_workspace(*a);
  if (need > 0 && (a->workspace == nullptr || a->workspace_bytes < need)) return GLU_EINVAL;
  Check c;
  c.matrix(a->x, a->M, a->K, a->ld_x);
  weights(c, a->w, a->E, a->N, a->K, a->ld_w, a->stride_w);
  c.matrix(a->residual, a->M, a->N, a->ld_residual);
  c.matrix(a->y, a->M, a->N, a->ld_y);
  c.matrix(a->z, a->M, a->N, a->ld_z);
  for (const void* p : {a->bias, static_cast<const void*>(a->offsets), static_cast<const void*>(a->workspace)}) c.vec(p);
  return c.status;
}

int check_linear_bwd(const glu_block_linear_bwd_args* a, bool query) {
  if (a == nullptr || a->act < GLU_ACT_SILU || a->act > GLU_ACT_GELU_ERF) return GLU_EINVAL;
  const int st = check_linear_size(a->M, a->N, a->K, a->E);
  if (st != GLU_OK) return st;
  if (query) return GLU_OK;
  if (!a->dy || (a->z != nullptr) != (a->act != GLU_ACT_IDENTITY) || (a->offsets != nullptr) != (a->E > 0)) return GLU_EINVAL;
  if ((!a->dx && !a->dw && !a->db) || (a->dx && !a->w) || (a->dw && !a->x)) return GLU_EINVAL;
  const size_t need = gq::linear_bwd_workspace(*a);
  if (need > 0 && (a->workspace == nullptr || a->workspace_bytes < need)) return GLU_EINVAL;
  Check c;
  c.matrix(a->dy, a->M, a->N, a->ld_dy);
  c.matrix(a->z, a->M, a->N, a->ld_z);
  if (a->dw) c.matrix(a->x, a->M, a->K, a->ld_x);
  if (a->dx) weights(c, a->w, a->E, a->N, a->K, a->ld_w, a->stride_w);
  c.matrix(a->dx, a->M, a->K, a->ld_dx);
  weights(c, a->dw, a->E, a->N, a->K, a->ld_dw, a->stride_dw);
  for (const void* p : {static_cast<const void*>(a->db), static_cast<const void*>(a->offsets), static_cast<const void*>(a->workspace)})
    c.vec(p);
  return c.status;
}

}  // namespace

// Every entry point: its checks, the device, the launch.
#define GQ_ENTRY(check, launch)                       \
  const int st = (check);                             \
  if (st != GLU_OK) return st;                        \
  gq::DevInfo d;                                      \
  const int dev = gq::device_info(&d);                \
  if (dev != GLU_OK) return dev;                      \
  const cudaStream_t s = static_cast<cudaStream_t>(stream); \
  return launched(launch)

extern "C" int glu_block_norm_fwd(const glu_block_norm_fwd_args* a, void* stream) {
  GQ_ENTRY(check_norm_fwd(a), gq::launch_norm_fwd(*a, s, d));
}
extern "C" int glu_block_norm_bwd(const glu_block_norm_bwd_args* a, void* stream) {
  GQ_ENTRY(check_norm_bwd(a), gq::launch_norm_bwd(*a, s));
}
extern "C" int glu_block_route(const glu_block_route_args* a, void* stream) {
  GQ_ENTRY(check_route(a), gq::launch_route(*a, s));
}
extern "C" int glu_block_dispatch(const glu_block_rows_args* a, void* stream) {
  GQ_ENTRY(check_rows(a, kDispatch), gq::launch_dispatch(*a, s, d));
}
extern "C" int glu_block_combine(const glu_block_rows_args* a, void* stream) {
  GQ_ENTRY(check_rows(a, kCombine), gq::launch_combine(*a, s, d));
}
extern "C" int glu_block_combine_bwd(const glu_block_rows_args* a, void* stream) {
  GQ_ENTRY(check_rows(a, kCombineBwd), gq::launch_combine_bwd(*a, s, d));
}
extern "C" int glu_block_linear_fwd(const glu_block_linear_fwd_args* a, void* stream) {
  GQ_ENTRY(check_linear_fwd(a, false), gq::launch_linear_fwd(*a, s, d));
}
extern "C" int glu_block_linear_bwd(const glu_block_linear_bwd_args* a, void* stream) {
  GQ_ENTRY(check_linear_bwd(a, false), gq::launch_linear_bwd(*a, s, d));
}

extern "C" int glu_block_norm_bwd_workspace(int64_t M, int64_t D, int64_t gates, size_t* bytes) {
  if (bytes == nullptr || M <= 0 || D <= 0 || gates < 0) return GLU_EINVAL;
  if (D > kMaxNormBwd || (gates > 0 && M % gates != 0)) return GLU_ESHAPE;
  *bytes = gq::norm_bwd_workspace(M, D, gates);
  return GLU_OK;
}
extern "C" int glu_block_route_workspace(int64_t T, int64_t K, int32_t E, size_t* bytes) {
  if (bytes == nullptr) return GLU_EINVAL;
  const int st = check_route_size(T, K, E);
  if (st == GLU_OK) *bytes = gq::route_workspace(T, K, E);
  return st;
}
extern "C" int glu_block_linear_fwd_workspace(const glu_block_linear_fwd_args* a, size_t* bytes) {
  if (bytes == nullptr) return GLU_EINVAL;
  const int st = check_linear_fwd(a, true);
  if (st == GLU_OK) *bytes = gq::linear_fwd_workspace(*a);
  return st;
}
extern "C" int glu_block_linear_bwd_workspace(const glu_block_linear_bwd_args* a, size_t* bytes) {
  if (bytes == nullptr) return GLU_EINVAL;
  const int st = check_linear_bwd(a, true);
  if (st == GLU_OK) *bytes = gq::linear_bwd_workspace(*a);
  return st;
}

extern "C" int glu_block_device_errors(uint32_t* bits, int clear) {
  if (bits == nullptr) return GLU_EINVAL;
  uint32_t norm = 0, linear8 = 0;
  if (gq::read_err_linear(bits, clear != 0) != cudaSuccess || gq::read_err_norm(&norm, clear != 0) != cudaSuccess ||
      gq::read_err_linear8(&linear8, clear != 0) != cudaSuccess) {
    cudaGetLastError();
    return GLU_EDEVICE;
  }
  *bits |= norm | linear8;
  return GLU_OK;
}
extern "C" int glu_block_abi_version(void) { return GLU_BLOCK_ABI_VERSION; }
