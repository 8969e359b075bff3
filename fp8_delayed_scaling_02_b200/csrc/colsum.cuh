// The second launch of a column sum: adds the rows that the blocks of the
// first one wrote, in a fixed order.
#pragma once

#include "common.cuh"

namespace fp8ds {
namespace {

// out[c] = sum over p of partial[p][c], p ascending within each of the 32
// warps of a block and the warps' sums in order.
__global__ void __launch_bounds__(1024) colsum_kernel(const float* partial, int n, int64_t cols, float* out) {
  __shared__ float s[32][33];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = int64_t(blockIdx.x) * 32 + lane;
  float acc = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int p = warp; p < n; p += 32) acc += partial[p * cols + c];
  }
  s[warp][lane] = acc;
  __syncthreads();
  if (warp == 0 && c < cols) {
    float r = 0.0f;
#pragma unroll
    for (int w = 0; w < 32; ++w) r += s[w][lane];
    out[c] = r;
  }
}

int launch_colsum(const float* partial, int n, int64_t cols, float* out, cudaStream_t st) {
  if (cols == 0) return FP8_OK;
  return launch_pdl(colsum_kernel, dim3(unsigned((cols + 31) / 32)), dim3(1024), 0, st, 1, partial, n, cols, out) ==
                 cudaSuccess
             ? FP8_OK
             : FP8_ERR_CUDA;
}

}  // namespace
}  // namespace fp8ds
