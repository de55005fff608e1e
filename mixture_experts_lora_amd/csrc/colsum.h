// Sums over blocks' float32 partial rows, the second pass of the gradients that are sums over tokens.
#pragma once

#include "device_common.h"

namespace moe {

// Column sum of part [groups][stride], for a block of 1024 threads and 32 columns from col0 on (a
// multiple of 4 of them exist, `cols` in all): 128 rows of 8 lanes, 16 bytes a lane, walk every
// 128th group with eight loads in flight; the 128 sums meet in LDS, in a fixed order. True for the
// 32 threads that get one, with its column.
__device__ __forceinline__ bool block_colsum(const float* part, int64_t groups, int64_t stride,
                                             int col0, int cols, float (&red)[128][33], int& col,
                                             float& total) {
  const int cx = threadIdx.x & 7, ry = threadIdx.x >> 3, c4 = col0 + cx * 4;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c4 < cols) {
#pragma unroll 8
    for (int64_t g = ry; g < groups; g += 128) {
      const float4 v = *reinterpret_cast<const float4*>(part + g * stride + c4);
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
  }
  red[ry][cx * 4] = a.x;
  red[ry][cx * 4 + 1] = a.y;
  red[ry][cx * 4 + 2] = a.z;
  red[ry][cx * 4 + 3] = a.w;
  __syncthreads();
  const int c = threadIdx.x & 31, row = threadIdx.x >> 5;
  total = (red[row][c] + red[row + 32][c]) + (red[row + 64][c] + red[row + 96][c]);
  __syncthreads();
  red[row][c] = total;
  __syncthreads();
  col = col0 + c;
  if (row != 0 || col >= cols) return false;
  total = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) total += red[i][c];
  return true;
}

}  // namespace moe
