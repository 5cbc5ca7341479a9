// Internal launcher interface of the block operators (glu_block.h) between
// the C-ABI layer (block_api.cu) and the kernel translation units.
// Arguments are already validated.
#pragma once

#include "glu_block.h"
#include "kernels.h"

namespace gq {

constexpr int kMaxExperts = 1024;

// The current device's facts; GLU_OK, or GLU_EDEVICE unless it is a GB300
// (api.cu).
int device_info(DevInfo* info);

// `count` row-major bf16 matrices of rows x cols, `stride_bytes` apart, loaded
// in boxes of 64 columns (128 bytes, the 128-byte swizzle) by box_rows rows of
// one matrix; what lies outside a matrix is filled with zeros (block_tmap.cu).
cudaError_t make_stack_map(CUtensorMap* map, const void* base, int64_t cols, int64_t rows, int64_t row_stride_bytes,
                           int64_t count, int64_t stride_bytes, int box_rows);

cudaError_t launch_norm_fwd(const glu_block_norm_fwd_args& a, cudaStream_t s, const DevInfo& d);
cudaError_t launch_norm_bwd(const glu_block_norm_bwd_args& a, cudaStream_t s);
cudaError_t read_err_norm(uint32_t* v, bool clear);
size_t norm_bwd_workspace(int64_t M, int64_t D, int64_t gates);

cudaError_t launch_route(const glu_block_route_args& a, cudaStream_t s);
size_t route_workspace(int64_t T, int64_t K, int32_t E);
cudaError_t launch_dispatch(const glu_block_rows_args& a, cudaStream_t s, const DevInfo& d);
cudaError_t launch_combine(const glu_block_rows_args& a, cudaStream_t s, const DevInfo& d);
cudaError_t launch_combine_bwd(const glu_block_rows_args& a, cudaStream_t s, const DevInfo& d);

cudaError_t launch_linear_fwd(const glu_block_linear_fwd_args& a, cudaStream_t s, const DevInfo& d);
cudaError_t launch_linear_bwd(const glu_block_linear_bwd_args& a, cudaStream_t s, const DevInfo& d);
size_t linear_fwd_workspace(const glu_block_linear_fwd_args& a);
size_t linear_bwd_workspace(const glu_block_linear_bwd_args& a);
cudaError_t read_err_linear(uint32_t* v, bool clear);

}  // namespace gq
