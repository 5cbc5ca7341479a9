// The sums over a block of one, two or three values, alone: for each number of
// warps what every thread gets from a call ahead of a loop and from each call
// inside it.  Values are whole numbers, so that the sums are exact.
#include <cuda_runtime.h>

#include "block_util.cuh"

namespace {

constexpr int kCalls = 4;  // one ahead of the loop, three in it

// Value j of thread t at call c; the test computes the same.
__device__ float value_of(int t, int j, int c) { return float((t * (2 * j + 1) + 7 * c + 3 * j) % 61); }

// out [kCalls][N][threads]
template <int N>
__global__ void __launch_bounds__(1024) sum_kernel(float* out, int calls) {
  __shared__ gq::BlockSum<N> sums;
  uint32_t buf = 0;
  const int threads = blockDim.x, t = threadIdx.x;
  float v[N];
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = value_of(t, j, 0);
  gq::block_sum(sums, buf, threads, v);
#pragma unroll
  for (int j = 0; j < N; ++j) out[j * threads + t] = v[j];
  for (int c = 1; c < calls; ++c) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = value_of(t, j, c);
    gq::block_sum(sums, buf, threads, v);
#pragma unroll
    for (int j = 0; j < N; ++j) out[(c * N + j) * threads + t] = v[j];
  }
}

}  // namespace

// Sums of n values over `warps` warps into host memory [4][n][32 * warps]; 0 on success.
extern "C" GLU_API int gq_probe_block_sum(int n, int warps, float* host) {
  if (n < 1 || n > 3 || warps < 1 || warps > (n == 1 ? 32 : 16)) return 1;
  const int threads = 32 * warps;
  const size_t bytes = size_t(kCalls) * n * threads * sizeof(float);
  float* d = nullptr;
  if (cudaMalloc(&d, bytes) != cudaSuccess) return 2;
  if (n == 1) sum_kernel<1><<<1, threads>>>(d, kCalls);
  if (n == 2) sum_kernel<2><<<1, threads>>>(d, kCalls);
  if (n == 3) sum_kernel<3><<<1, threads>>>(d, kCalls);
  const bool ok = cudaGetLastError() == cudaSuccess && cudaMemcpy(host, d, bytes, cudaMemcpyDeviceToHost) == cudaSuccess;
  return cudaFree(d) == cudaSuccess && ok ? 0 : 3;
}
