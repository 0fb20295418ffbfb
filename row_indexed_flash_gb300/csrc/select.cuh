// Selection helpers shared by the block and eviction selections: an
// order-preserving key of a score and block-wide prefix sums.
#pragma once

#include "fa_internal.cuh"

namespace far {

// Larger score -> larger key, at least 2; a NaN takes 1, below every number;
// 0 is left for entries that cannot be chosen.  -0 and +0 are one value.
__device__ __forceinline__ uint32_t score_key(float x) {
  const uint32_t u = __float_as_uint(x);
  if (x != x) return 1u;
  if (x == 0.f) return 0x80000000u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);   // -inf -> 0x007fffff
}

// Exclusive prefix sum of v over a block of NT threads; *total gets the sum.
// warp_sums: NT / 32 ints of shared memory.
template <int NT>
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  constexpr int NW = NT / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const int t = warp_sums[w];
    before += w < warp ? t : 0;
    sum += t;
  }
  *total = sum;
  __syncthreads();
  return before + x - v;
}

}  // namespace far
