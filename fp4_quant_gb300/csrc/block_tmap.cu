// TMA descriptors of stacks of matrices (the linear layers' weights by expert).
#include <atomic>
#include <cudaTypedefs.h>

#include "block8.h"

namespace gq {
namespace {

std::atomic<PFN_cuTensorMapEncodeTiled_v12000> g_encode{nullptr};

// The driver's encoder, looked up once through the runtime.
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  PFN_cuTensorMapEncodeTiled_v12000 f = g_encode.load(std::memory_order_acquire);
  if (f != nullptr) return f;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess || fn == nullptr) {
    cudaGetLastError();
    return nullptr;
  }
  f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  g_encode.store(f, std::memory_order_release);
  return f;
}

}  // namespace

static cudaError_t stack_map(CUtensorMap* map, CUtensorMapDataType type, int box_cols, const void* base, int64_t cols, int64_t rows,
                             int64_t row_stride_bytes, int64_t count, int64_t stride_bytes, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (enc == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(count)};
  const cuuint64_t strides[2] = {cuuint64_t(row_stride_bytes), cuuint64_t(stride_bytes)};
  const cuuint32_t box[3] = {cuuint32_t(box_cols), cuuint32_t(box_rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, type, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t make_stack_map(CUtensorMap* map, const void* base, int64_t cols, int64_t rows, int64_t row_stride_bytes,
                           int64_t count, int64_t stride_bytes, int box_rows) {
  return stack_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 64, base, cols, rows, row_stride_bytes, count, stride_bytes, box_rows);
}

cudaError_t make_byte_stack_map(CUtensorMap* map, const void* base, int64_t cols, int64_t rows, int64_t row_stride, int64_t count,
                                int64_t stride, int box_rows) {
  return stack_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 128, base, cols, rows, row_stride, count, stride, box_rows);
}

}  // namespace gq
