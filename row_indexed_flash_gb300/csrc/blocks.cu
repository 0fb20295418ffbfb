// Operators on 64-row blocks (pages) of keys: their elementwise bounds, the
// bound of a query's logits over a block, and the row lists of chosen blocks.
#include <string.h>

#include "blocks.cuh"
#include "keyscan.cuh"
#include "kvread.cuh"
#include "select.cuh"

namespace far {

namespace {

// ---------------------------------------------------------------------------
// Bounds: kmin[page, g, d], kmax[page, g, d] over the page's first fill rows.
// HBM-bound: each key is read once.  A page is 64 rows of Hkv * D contiguous
// elements; a thread owns one 16-byte column of it and up to 8 of its rows, all
// loaded before any is looked at, and a CTA's row groups meet in shared memory.
// 16-bit pools are compared as they stand, two columns an instruction; codes
// of quantised pools as code * scale in fp32 (exact), two rows a comparison,
// rounded outward at the end.  A NaN key makes its bounds NaN.  Measured for
// 1,562 pages of 8 heads, D 128: bf16 35 us (5.97 TB/s, 0.88 of the copy rate),
// INT8 34 us (3.2 TB/s: the ALU, at 56 %, and the issue slots, at 63 %, hold
// it), INT4 37 us, E4M3 38 us; 32 pages 2.7 us.

constexpr int kBndThreads = 256;
constexpr int kBndRows = 8;   // rows per thread

__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float y;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// A 16-byte load that stays where it is written: a thread's loads all go out
// before the first is used (left to itself the compiler uses each at once).
__device__ __forceinline__ uint4 load_in_order(const void* p) {
  uint4 w;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(p));
  return w;
}
__device__ __forceinline__ uint16_t round16(float x, bool up, bool bf16) {
  if (bf16) return __bfloat16_as_ushort(up ? __float2bfloat16_ru(x) : __float2bfloat16_rd(x));
  return __half_as_ushort(up ? __float2half_ru(x) : __float2half_rd(x));
}
template <int KIND>
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  if constexpr (KIND == KV_BF16) {
    const __nv_bfloat162 y = __hmin2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&y);
  } else {
    const __half2 y = __hmin2_nan(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&y);
  }
}
template <int KIND>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  if constexpr (KIND == KV_BF16) {
    const __nv_bfloat162 y = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&y);
  } else {
    const __half2 y = __hmax2_nan(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&y);
  }
}

template <int KIND>
__global__ void __launch_bounds__(kBndThreads) bounds_kernel(const BoundsParams p, int cx) {
  constexpr bool QUANT = KIND == KV_I8 || KIND == KV_I4 || KIND == KV_F8;
  constexpr int N = KvChunk<KIND>::N;            // elements of a column
  constexpr int W = QUANT ? N : N / 2;           // words that hold one bound of a column
  extern __shared__ uint32_t bsm[];              // [row group][cx][2 W (+ 1)]
  const int page = __ldg(p.pages + blockIdx.x);
  if (page < 0 || (long long)page >= p.n_pool_pages) return;
  const int fill = p.fill ? min(max(__ldg(p.fill + blockIdx.x), 0), kPage) : kPage;
  if (fill == 0) return;
  const int rb = kv_row_bytes<KIND>(p.D);
  const int cpr = p.Hkv * (rb / 16);             // 16-byte columns of a row
  const int x = threadIdx.x % cx, rg = threadIdx.x / cx, nrg = kBndThreads / cx;
  const int col = blockIdx.y * cx + x;
  const float INF = __int_as_float(0x7f800000);
  uint32_t lo[W], hi[W];
#pragma unroll
  for (int t = 0; t < W; ++t) {
    lo[t] = QUANT ? 0x7f800000u : KIND == KV_BF16 ? 0x7f807f80u : 0x7c007c00u;   // +inf
    hi[t] = lo[t] | (QUANT ? 0x80000000u : 0x80008000u);
  }
  if (col < cpr) {
    const char* src = static_cast<const char*>(p.k) + ((size_t)page * kPage * cpr + col) * 16;
    const uint16_t* sc = QUANT ? p.k_scale + ((size_t)page * p.Hkv + col / (rb / 16)) * kPage : nullptr;
    // rows rg, rg + nrg, ...; a row past the fill is replaced by row 0, which
    // the bounds hold anyway
    uint4 w[kBndRows];
    unsigned short s16[kBndRows];
#pragma unroll
    for (int i = 0; i < kBndRows; ++i) {
      const int r = rg + i * nrg < fill ? rg + i * nrg : 0;
      w[i] = load_in_order(src + (size_t)r * cpr * 16);
      if (QUANT) s16[i] = __ldg(sc + r);
    }
    if constexpr (QUANT) {
#pragma unroll
      for (int i = 0; i < kBndRows; i += 2) {
        float a[N], b[N];
        kv_codes<KIND>(w[i], a);
        kv_codes<KIND>(w[i + 1], b);
        const float sa = __half2float(__ushort_as_half(s16[i])), sb = __half2float(__ushort_as_half(s16[i + 1]));
#pragma unroll
        for (int t = 0; t < N; t += 2) {
          const float2 va = __fmul2_rn(make_float2(a[t], a[t + 1]), make_float2(sa, sa));
          const float2 vb = __fmul2_rn(make_float2(b[t], b[t + 1]), make_float2(sb, sb));
          lo[t] = __float_as_uint(min3_nan(__uint_as_float(lo[t]), va.x, vb.x));
          hi[t] = __float_as_uint(max3_nan(__uint_as_float(hi[t]), va.x, vb.x));
          lo[t + 1] = __float_as_uint(min3_nan(__uint_as_float(lo[t + 1]), va.y, vb.y));
          hi[t + 1] = __float_as_uint(max3_nan(__uint_as_float(hi[t + 1]), va.y, vb.y));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kBndRows; ++i) {
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int t = 0; t < W; ++t) {
          lo[t] = min2_nan<KIND>(lo[t], u[t]);
          hi[t] = max2_nan<KIND>(hi[t], u[t]);
        }
      }
    }
  }
  uint32_t* mine = bsm + (size_t)threadIdx.x * (2 * W + 1);
#pragma unroll
  for (int t = 0; t < W; ++t) {
    mine[t] = lo[t];
    mine[W + t] = hi[t];
  }
  __syncthreads();
  // one word of one column's bounds per thread, over the row groups that hold rows
  const int groups = min(nrg, kPage);
  for (int f = threadIdx.x; f < cx * W; f += kBndThreads) {
    const int xx = f / W, t = f % W, cc = blockIdx.y * cx + xx;
    if (cc >= cpr) continue;
    uint32_t l = bsm[(size_t)xx * (2 * W + 1) + t], h = bsm[(size_t)xx * (2 * W + 1) + W + t];
    for (int r = 1; r < groups; ++r) {
      const uint32_t* o = bsm + (size_t)(r * cx + xx) * (2 * W + 1);
      if constexpr (QUANT) {
        l = __float_as_uint(min3_nan(__uint_as_float(l), __uint_as_float(o[t]), INF));
        h = __float_as_uint(max3_nan(__uint_as_float(h), __uint_as_float(o[W + t]), -INF));
      } else {
        l = min2_nan<KIND>(l, o[t]);
        h = max2_nan<KIND>(h, o[W + t]);
      }
    }
    const size_t at = ((size_t)page * cpr + cc) * W + t;   // words of 2 (16-bit pools) or elements
    if constexpr (QUANT) {
      static_cast<uint16_t*>(p.kmin)[at] = round16(__uint_as_float(l), false, p.out_bf16);
      static_cast<uint16_t*>(p.kmax)[at] = round16(__uint_as_float(h), true, p.out_bf16);
    } else {
      static_cast<uint32_t*>(p.kmin)[at] = l;
      static_cast<uint32_t*>(p.kmax)[at] = h;
    }
  }
}

template <int KIND>
cudaError_t bounds_kind(const BoundsParams& p, cudaStream_t st) {
  constexpr bool QUANT = KIND == KV_I8 || KIND == KV_I4 || KIND == KV_F8;
  constexpr int W = QUANT ? KvChunk<KIND>::N : KvChunk<KIND>::N / 2;
  const int cpr = p.Hkv * (kv_row_bytes<KIND>(p.D) / 16);
  // columns of a CTA: 32, or the row's own number rounded up to a power of two
  // (no fewer than 4: 64 row groups of one row each)
  int cx = 4;
  while (cx < cpr && cx < 32) cx <<= 1;
  const dim3 grid(p.n_pages, (cpr + cx - 1) / cx);
  const size_t smem = (size_t)kBndThreads * (2 * W + 1) * sizeof(uint32_t);
  const cudaError_t e = once_per_device<2>([smem] {
    return cudaFuncSetAttribute(bounds_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  bounds_kernel<KIND><<<grid, kBndThreads, smem, st>>>(p, cx);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Block rows: one CTA per (slice, KV head).  The k-th largest key among the
// middle blocks by histograms over the keys' range, then one ordered pass that
// writes the chosen blocks' rows.  Bound by latency: 32 x 8 lists of 32 of up
// to 2,048 blocks 8 us.

constexpr int kBrThreads = 512;
constexpr int kBrWarps = kBrThreads / 32;
constexpr int kBrPer = 4;              // consecutive blocks per thread and step
constexpr int kBrCap = 32768;          // blocks whose keys are kept in shared memory

__global__ void __launch_bounds__(kBrThreads) block_rows_kernel(const BlockRowsParams p, int cap) {
  extern __shared__ uint32_t keys[];   // [cap]
  __shared__ int hist[kBrThreads];
  __shared__ uint32_t ends[2];         // smallest and largest key of the middle
  __shared__ int warp_sums[kBrWarps + 1];
  __shared__ int state[3];
  __shared__ int last_listed;          // whether the sequence's last block was chosen
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.x, s = blockIdx.y;
  if (tid == 0) {
    last_listed = 0;
    ends[0] = 0xffffffffu;
    ends[1] = 0u;
  }
  const int seq = p.slice_seq ? __ldg(p.slice_seq + s) : s;
  const bool seq_ok = seq >= 0 && seq < p.n_seq;
  const long long cap_rows = (long long)p.max_pages * kPage;
  long long n = seq_ok ? max(__ldg(p.seq_len + s), 0) : 0;
  if (n > cap_rows) n = cap_rows;
  const int nb = (int)((n + kPage - 1) / kPage);
  const int lo = min(p.sinks, nb), hi = max(lo, nb - p.recent);
  const int m = hi - lo, kk = min(p.k, m);
  const bool take_all = kk == m;
  const float* sc = p.score + ((size_t)s * p.Hkv + g) * p.max_pages;
  const int32_t* table = p.page_table + (size_t)(seq_ok ? seq : 0) * p.max_pages;
  int32_t* out = p.kv_rows + ((size_t)s * p.Hkv + g) * p.list_len;
  auto key_at = [&](int b) { return b < cap ? keys[b] : score_key(__ldg(sc + b)); };

  KeyRange range = key_range(0u, 0u, kk);
  if (!take_all && kk > 0) {
    __syncthreads();
    uint32_t kmin = 0xffffffffu, kmax = 0u;
    for (int b = lo + tid; b < hi; b += kBrThreads) {
      const uint32_t key = score_key(__ldg(sc + b));
      if (b < cap) keys[b] = key;
      kmin = min(kmin, key);
      kmax = max(kmax, key);
    }
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    if (lane == 0) {
      atomicMin(&ends[0], kmin);
      atomicMax(&ends[1], kmax);
    }
    __syncthreads();
    range = key_range(ends[0], ends[1], kk);
    while (!range.done) {
      hist[tid] = 0;
      __syncthreads();
      const int shift = range_shift<kBrThreads>(range);
      for (int b = lo + tid; b < hi; b += kBrThreads) {
        const uint32_t key = key_at(b);
        if (in_range(range, key)) atomicAdd(&hist[(key - range.base) >> shift], 1);
      }
      __syncthreads();
      range_pick<kBrThreads>(range, hist[kBrThreads - 1 - tid], warp_sums, state);
      __syncthreads();   // state and hist may be written again
    }
  }
  const uint32_t T = range.T;
  const int need_eq = range.need_eq;

  // chosen blocks in order; out_at = blocks listed before this step
  int out_at = 0, eq_seen = 0;
  for (int base = 0; base < nb; base += kBrThreads * kBrPer) {
    const int b0 = base + tid * kBrPer;
    uint32_t key[kBrPer];
    int n_eq = 0;
#pragma unroll
    for (int u = 0; u < kBrPer; ++u) {
      const int b = b0 + u;
      key[u] = 0u;
      if (b >= lo && b < hi && !take_all && kk > 0) {
        key[u] = key_at(b);
        n_eq += key[u] == T;
      }
    }
    int eq_total = 0;
    int eq = eq_seen + block_scan<kBrThreads>(n_eq, warp_sums, &eq_total);
    unsigned sel = 0u;
#pragma unroll
    for (int u = 0; u < kBrPer; ++u) {
      const int b = b0 + u;
      bool on = b < lo || (b >= hi && b < nb);
      if (b >= lo && b < hi) {
        on = take_all;
        if (!take_all && kk > 0) {
          on = key[u] > T;
          if (key[u] == T) on = eq++ < need_eq;
        }
      }
      sel |= (on ? 1u : 0u) << u;
      if (on && b == nb - 1) last_listed = 1;
    }
    int total = 0;
    const int at = out_at + block_scan<kBrThreads>(__popc(sel), warp_sums, &total);
    // the warp writes the 64 rows of each of its chosen blocks together
#pragma unroll
    for (int u = 0; u < kBrPer; ++u) {
      const unsigned who = __ballot_sync(0xffffffffu, (sel >> u) & 1u);
      const int my_at = at + __popc(sel & ((1u << u) - 1u));
      const int my_page = (sel >> u) & 1u ? __ldg(table + b0 + u) : -1;
      for (unsigned w = who; w; w &= w - 1) {
        const int l = __ffs(w) - 1;
        const int a = __shfl_sync(0xffffffffu, my_at, l), page = __shfl_sync(0xffffffffu, my_page, l);
        const int b = base + (warp * 32 + l) * kBrPer + u;
        const bool ok = page >= 0 && page <= (0x7fffffff - (kPage - 1)) / kPage;
#pragma unroll
        for (int t = lane; t < kPage; t += 32) {
          const bool in = (long long)b * kPage + t < n;
          out[(size_t)a * kPage + t] = ok && in ? page * kPage + t : -1;
        }
      }
    }
    out_at += total;
    eq_seen += eq_total;
  }
  // entries: whole blocks, but for the sequence's last one where it is listed
  for (int j = out_at * kPage + tid; j < p.list_len; j += kBrThreads) out[j] = -1;
  __syncthreads();
  if (tid == 0) {
    int len = out_at * kPage;
    if (last_listed) len -= nb * kPage - (int)n;
    p.kv_len[(size_t)s * p.Hkv + g] = len;
  }
}

}  // namespace

cudaError_t bounds_launch(const BoundsParams& p, cudaStream_t st) {
  switch (p.kind) {
    case KV_BF16: return bounds_kind<KV_BF16>(p, st);
    case KV_F16: return bounds_kind<KV_F16>(p, st);
    case KV_I8: return bounds_kind<KV_I8>(p, st);
    case KV_I4: return bounds_kind<KV_I4>(p, st);
    case KV_F8: return bounds_kind<KV_F8>(p, st);
  }
  return cudaErrorInvalidValue;
}

cudaError_t scores_launch(const ScoresParams& p, cudaStream_t st) {
  KeyScanParams k;
  memset(&k, 0, sizeof(k));
  k.q = p.q;
  k.k[0] = p.kmax;
  k.k[1] = p.kmin;
  k.rows = p.page_table;
  k.len = p.seq_len;
  k.slice_seq = p.slice_seq;
  k.out = p.score;
  k.R = p.n_pool_pages;
  k.S = p.S;
  k.Nq = p.Nq;
  k.Hq = p.Hq;
  k.Hkv = p.Hkv;
  k.L = p.max_pages;
  k.G = p.G;
  k.NV = p.Nq * p.G;
  k.n_seq = p.n_seq;
  k.q_bf16 = p.q_bf16;
  k.err = p.err;
  k.wait_ns = p.wait_ns;
  return keyscan_scores(k, p.D, st);
}

cudaError_t block_rows_launch(const BlockRowsParams& p, cudaStream_t st) {
  const int cap = p.max_pages < kBrCap ? p.max_pages : kBrCap;
  const cudaError_t e = once_per_device<1>(
      [] { return cudaFuncSetAttribute(block_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBrCap * 4); });
  if (e != cudaSuccess) return e;
  block_rows_kernel<<<dim3(p.Hkv, p.S), kBrThreads, (size_t)cap * 4, st>>>(p, cap);
  return cudaGetLastError();
}

}  // namespace far
