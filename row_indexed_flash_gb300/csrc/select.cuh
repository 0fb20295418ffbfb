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
// warp_sums: NT / 32 + 1 ints of shared memory.
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
  if (warp == 0) {
    const int own = lane < NW ? warp_sums[lane] : 0;
    int w = own;
#pragma unroll
    for (int o = 1; o < NW; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    if (lane < NW) warp_sums[lane] = w - own;
    if (lane == NW - 1) warp_sums[NW] = w;
  }
  __syncthreads();
  const int before = warp_sums[warp] + x - v;
  *total = warp_sums[NW];
  __syncthreads();
  return before;
}

// Selection of the k-th largest of many 32-bit keys by histograms over the
// keys' own range: the range [base, base + 2^bits) of the keys still in
// question is cut into NT bins, the bin that holds the k-th largest becomes
// the next range.  Cutting the range that is there, not fixed digits of the
// key, spreads the first histogram (the upper digits of float scores are
// nearly all alike, and their atomics would queue), so that two or three
// passes do.
struct KeyRange {
  uint32_t base;   // first key of the range
  int bits;        // its width: keys with (key - base) >> bits == 0
  int left;        // how many of its keys, from the top, are still to take
  bool done;       // threshold and need_eq are final
  uint32_t T;      // keys above T are taken ...
  int need_eq;     // ... and the first need_eq equal to it
};

__device__ __forceinline__ KeyRange key_range(uint32_t kmin, uint32_t kmax, int k) {
  KeyRange r;
  r.base = kmin;
  r.bits = 32 - __clz((int)(kmax - kmin));
  r.left = k;
  r.done = false;
  r.T = 0xffffffffu;
  r.need_eq = 0;
  return r;
}
template <int NT>
__device__ __forceinline__ int range_shift(const KeyRange& r) {
  constexpr int LOG = NT == 1024 ? 10 : NT == 512 ? 9 : 8;
  static_assert((1 << LOG) == NT, "bins");
  return max(r.bits - LOG, 0);
}
__device__ __forceinline__ bool in_range(const KeyRange& r, uint32_t key) {
  return r.bits >= 32 || ((key - r.base) >> r.bits) == 0u;
}
// Narrows the range to the bin where the count from the top reaches `left`.
// Thread t brings the count of bin NT - 1 - t.  state: 3 ints of shared memory.
template <int NT>
__device__ __forceinline__ void range_pick(KeyRange& r, int count, int* warp_sums, int* state) {
  int total;
  const int above = block_scan<NT>(count, warp_sums, &total);
  if (above < r.left && above + count >= r.left) {
    state[0] = NT - 1 - (int)threadIdx.x;
    state[1] = r.left - above;
    state[2] = count;
  }
  __syncthreads();
  const int shift = range_shift<NT>(r);
  r.base += (uint32_t)state[0] << shift;
  r.left = state[1];
  r.bits = shift;
  if (state[2] == r.left) {          // the whole bin: every key from base on
    r.T = r.base - 1u;
    r.done = true;
  } else if (shift == 0) {           // one key value, some of its holders
    r.T = r.base;
    r.need_eq = r.left;
    r.done = true;
  }
}

}  // namespace far
