// column_sum.h -- sums over the rows of a matrix of partial sums, for the
// gradients of parameters (gfx950).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ssm {

constexpr int kSumThreads = 1024;

// Sum of `rows` rows of `cols` floats at column col (of the calling thread; 32
// neighbouring columns a workgroup of kSumThreads, 32 threads a column), in 64
// bits and a fixed order: a thread takes every 32nd row, eight loads in flight,
// then the threads' sums are added.  Valid in threads 0 .. 31.  (Four threads a
// column left a CU with as many loads as one wave has: 20 us for 1024 x 2560,
// 5 us so.)
__device__ __forceinline__ double column_sum(const float *part, int64_t rows, int64_t cols, int64_t col) {
  __shared__ double room[kSumThreads / 64][32];
  const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
  double v = 0.0;
  if (col < cols) {
    int64_t r = q;
    for (; r + 7 * 32 < rows; r += 8 * 32) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = part[(r + i * 32) * cols + col];
#pragma unroll
      for (int i = 0; i < 8; ++i) v += f[i];
    }
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = r + i * 32 < rows ? part[(r + i * 32) * cols + col] : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += f[i];
  }
  v += __shfl_xor(v, 32);
  if ((threadIdx.x & 32) == 0) room[threadIdx.x >> 6][lane] = v;
  __syncthreads();
  if (threadIdx.x >= 32) return 0.0;
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < kSumThreads / 64; ++k) s += room[k][lane];
  return s;
}

}  // namespace ssm
