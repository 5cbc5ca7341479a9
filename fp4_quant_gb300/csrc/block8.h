// Internal launcher interface of the operators in 8 bits (glu_block8.h)
// between the C-ABI layer (block8_api.cu) and the kernel translation units.
// Arguments are already validated.
#pragma once

#include "block.h"
#include "glu_block8.h"

namespace gq {

constexpr int kBlock8 = 128;  // values that share a scale along one dimension

inline int64_t blocks8(int64_t n) { return (n + kBlock8 - 1) / kBlock8; }
// Blocks of a column form.
inline int64_t col_blocks8(int64_t M, int32_t E) { return E > 0 ? M / kBlock8 + E : blocks8(M); }

// `count` row-major matrices of bytes, rows x cols, stride_bytes apart, loaded in
// boxes of 128 columns (the 128-byte swizzle) by box_rows rows of one matrix;
// what lies outside a matrix is filled with zeros (block_tmap.cu).
cudaError_t make_byte_stack_map(CUtensorMap* map, const void* base, int64_t cols, int64_t rows, int64_t row_stride, int64_t count,
                                int64_t stride, int box_rows);

cudaError_t launch_quant8(const glu_block8_quant_args& a, cudaStream_t s, const DevInfo& d);
cudaError_t launch_quant8_weight(const glu_block8_quant_weight_args& a, cudaStream_t s);
cudaError_t launch_glu8(const glu_block8_glu_args& a, cudaStream_t s);
cudaError_t launch_glu8_bwd(const glu_block8_glu_bwd_args& a, cudaStream_t s, const DevInfo& d);
cudaError_t launch_linear8(const glu_block8_linear_args& a, cudaStream_t s, const DevInfo& d);
// y of few tokens: the weights are read once (block8_linear_few.cu).
bool linear8_few(const glu_block8_linear_args& a);
cudaError_t launch_linear8_few(const glu_block8_linear_args& a, cudaStream_t s);
size_t linear8_workspace(const glu_block8_linear_args& a);
cudaError_t launch_linear8_dw(const glu_block8_linear_dw_args& a, cudaStream_t s, const DevInfo& d);
size_t linear8_dw_workspace(const glu_block8_linear_dw_args& a);
cudaError_t read_err_linear8(uint32_t* v, bool clear);

}  // namespace gq
