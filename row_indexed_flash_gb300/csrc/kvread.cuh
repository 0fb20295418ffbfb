// Reading pool elements as fp32, 16 bytes of one (row, KV head) at a time.
#pragma once

#include "fa_internal.cuh"
#include "widen.cuh"

namespace far {

// Bytes of one (pool row, KV head).
template <int KIND>
__host__ __device__ constexpr int kv_row_bytes(int D) {
  return KIND == KV_BF16 || KIND == KV_F16 ? 2 * D : KIND == KV_I4 ? D / 2 : D;
}
inline int kv_row_bytes(int kind, int D) {
  return kind == KV_BF16 || kind == KV_F16 ? 2 * D : kind == KV_I4 ? D / 2 : D;
}

// Elements in a 16-byte chunk.
template <int KIND>
struct KvChunk {
  static constexpr int N = KIND == KV_BF16 || KIND == KV_F16 ? 8 : KIND == KV_I4 ? 32 : 16;
};

// Scale of (row, head g) in the [R/64, Hkv, 64] layout.
__device__ __forceinline__ float kv_scale_of(const uint16_t* scale, int row, int g, int Hkv) {
  return __half2float(__ushort_as_half(__ldg(scale + ((size_t)(row >> 6) * Hkv + g) * kPage + (row & 63))));
}

// The fp32 codes of a 16-byte word (the values themselves for 16-bit pools).
template <int KIND>
__device__ __forceinline__ void kv_codes(const uint4& w, float (&x)[KvChunk<KIND>::N]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if constexpr (KIND == KV_BF16) {
      x[2 * t] = bf16_lo(u[t]);
      x[2 * t + 1] = bf16_hi(u[t]);
    } else if constexpr (KIND == KV_F16) {
      const float2 f = f16x2_to_f2(u[t]);
      x[2 * t] = f.x;
      x[2 * t + 1] = f.y;
    } else if constexpr (KIND == KV_I8) {
#pragma unroll
      for (int b = 0; b < 4; ++b) x[4 * t + b] = i8_to_f(u[t] ^ 0x80808080u, b);
    } else if constexpr (KIND == KV_F8) {
      const uint2 h = widen_e4m3x4(u[t]);
      const float2 lo = f16x2_to_f2(h.x), hi = f16x2_to_f2(h.y);
      x[4 * t] = lo.x;
      x[4 * t + 1] = lo.y;
      x[4 * t + 2] = hi.x;
      x[4 * t + 3] = hi.y;
    } else {
      const uint4 h = widen_i4x8(u[t], false);
      const uint32_t hv[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float2 f = f16x2_to_f2(hv[b]);
        x[8 * t + 2 * b] = f.x;
        x[8 * t + 2 * b + 1] = f.y;
      }
    }
  }
}

// Chunk c of (row r, head g): values (codes times scale, exact in fp32); zeros
// when r is negative (nothing is read).
template <int KIND>
__device__ __forceinline__ void kv_chunk(const void* pool, const uint16_t* scale, int r, int g, int Hkv, int D, int c,
                                         float (&x)[KvChunk<KIND>::N]) {
  if (r < 0) {
#pragma unroll
    for (int t = 0; t < KvChunk<KIND>::N; ++t) x[t] = 0.f;
    return;
  }
  const char* src = static_cast<const char*>(pool) + ((size_t)r * Hkv + g) * kv_row_bytes<KIND>(D) + c * 16;
  kv_codes<KIND>(__ldg(reinterpret_cast<const uint4*>(src)), x);
  if constexpr (KIND == KV_I8 || KIND == KV_I4 || KIND == KV_F8) {
    const float sc = kv_scale_of(scale, r, g, Hkv);
#pragma unroll
    for (int t = 0; t < KvChunk<KIND>::N; ++t) x[t] *= sc;
  }
}

}  // namespace far
