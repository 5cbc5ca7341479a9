// Between the products of the linear layers (block_linear.cu) and what stands
// around them (block_linear_rows.cu): few tokens, the join of split sums, and
// dz with its sums.
#pragma once

#include "block.h"

namespace gq {

// y of few tokens: the weights are read once, straight into registers.
bool linear_few(const glu_block_linear_fwd_args& a);
cudaError_t launch_linear_few(const glu_block_linear_fwd_args& a, cudaStream_t s);

// y (and z) from the fp32 parts [splits, M, N up to a multiple of 8] of z.
cudaError_t launch_linear_join(const glu_block_linear_fwd_args& a, const float* part, int splits, cudaStream_t s);

constexpr int kDzRows = 128;  // rows of one expert per block

struct DzP {
  const uint16_t *dy, *z;
  uint16_t* dz;  // NULL: not stored
  float* part;   // [slots, N], or NULL
  float* db;
  const int32_t* offsets;
  int64_t ld_dy, ld_z, ld_dz;
  int32_t rows, N, E, slots;
};

cudaError_t launch_linear_dz(int act, const DzP& p, cudaStream_t s);

}  // namespace gq
