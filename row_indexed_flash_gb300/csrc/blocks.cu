// Operators on 64-row blocks (pages) of keys: their elementwise bounds, the
// bound of a query's logits over a block, and the row lists of chosen blocks.
#include <string.h>

#include "blocks.cuh"
#include "keyscan.cuh"
#include "kvread.cuh"
#include "select.cuh"

namespace far {

namespace {

__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// ---------------------------------------------------------------------------
// Bounds: kmin[page, g, d], kmax[page, g, d] over the page's first fill rows.
// A page is 64 rows of Hkv * D contiguous elements, so a thread owns one
// 16-byte column of it and walks rows; the 8 row groups of a CTA meet in
// shared memory.  Rounded outward (exact for 16-bit pools).  A NaN key makes
// its bounds NaN.

constexpr int kBndThreads = 256;

__device__ __forceinline__ uint16_t round16(float x, bool up, bool bf16) {
  if (bf16) return __bfloat16_as_ushort(up ? __float2bfloat16_ru(x) : __float2bfloat16_rd(x));
  return __half_as_ushort(up ? __float2half_ru(x) : __float2half_rd(x));
}

template <int KIND>
__global__ void __launch_bounds__(kBndThreads) bounds_kernel(const BoundsParams p, int cx) {
  constexpr int N = KvChunk<KIND>::N;
  extern __shared__ float bsm[];   // [row group][cx][2 N]
  const int page = __ldg(p.pages + blockIdx.x);
  if (page < 0 || (long long)page >= p.n_pool_pages) return;
  const int fill = p.fill ? min(max(__ldg(p.fill + blockIdx.x), 0), kPage) : kPage;
  if (fill == 0) return;
  const int rb = kv_row_bytes<KIND>(p.D);
  const int cpr = p.Hkv * rb / 16;                 // 16-byte columns of a row
  const int x = threadIdx.x % cx, rg = threadIdx.x / cx, nrg = kBndThreads / cx;
  const int col = blockIdx.y * cx + x;
  const float INF = __int_as_float(0x7f800000);
  float lo[N], hi[N];
#pragma unroll
  for (int t = 0; t < N; ++t) {
    lo[t] = INF;
    hi[t] = -INF;
  }
  if (col < cpr) {
    const int g = col * 16 / rb, c = col - g * (rb / 16);
    for (int r = rg; r < fill; r += nrg) {
      float v[N];
      kv_chunk<KIND>(p.k, p.k_scale, page * kPage + r, g, p.Hkv, p.D, c, v);
#pragma unroll
      for (int t = 0; t < N; ++t) {
        lo[t] = min_nan(lo[t], v[t]);
        hi[t] = max_nan(hi[t], v[t]);
      }
    }
  }
  float* mine = bsm + (size_t)threadIdx.x * (2 * N + 1);
#pragma unroll
  for (int t = 0; t < N; ++t) {
    mine[t] = lo[t];
    mine[N + t] = hi[t];
  }
  __syncthreads();
  // thread -> one element of one bound of the slab
  for (int f = threadIdx.x; f < cx * N; f += kBndThreads) {
    const int xx = f / N, t = f % N;
    const int cc = blockIdx.y * cx + xx;
    if (cc >= cpr) continue;
    float l = INF, h = -INF;
    for (int r = 0; r < nrg; ++r) {
      const float* o = bsm + (size_t)(r * cx + xx) * (2 * N + 1);
      l = min_nan(l, o[t]);
      h = max_nan(h, o[N + t]);
    }
    const size_t at = (size_t)page * p.Hkv * p.D + (size_t)cc * N + t;
    static_cast<uint16_t*>(p.kmin)[at] = round16(l, false, p.out_bf16);
    static_cast<uint16_t*>(p.kmax)[at] = round16(h, true, p.out_bf16);
  }
}

template <int KIND>
cudaError_t bounds_kind(const BoundsParams& p, cudaStream_t st) {
  const int cpr = p.Hkv * kv_row_bytes<KIND>(p.D) / 16;
  int cx = 1;
  while (cx < cpr && cx < 32) cx <<= 1;
  const dim3 grid(p.n_pages, (cpr + cx - 1) / cx);
  const size_t smem = (size_t)kBndThreads * (2 * KvChunk<KIND>::N + 1) * sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(bounds_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  bounds_kernel<KIND><<<grid, kBndThreads, smem, st>>>(p, cx);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Block rows: one CTA per (slice, KV head).  The k-th largest key among the
// middle blocks by radix selection (four 8-bit digits, a histogram per warp),
// then one ordered pass that writes the chosen blocks' rows.

constexpr int kBrThreads = 512;
constexpr int kBrWarps = kBrThreads / 32;
constexpr int kBrPer = 4;              // consecutive blocks per thread and step
constexpr int kBrCap = 32768;          // blocks whose keys are kept in shared memory

__global__ void __launch_bounds__(kBrThreads) block_rows_kernel(const BlockRowsParams p, int cap) {
  extern __shared__ uint32_t keys[];   // [cap]
  __shared__ int hist[kBrWarps][256];
  __shared__ int warp_sums[kBrWarps];
  __shared__ int state[2];
  __shared__ int last_listed;          // whether the sequence's last block was chosen
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.x, s = blockIdx.y;
  if (tid == 0) last_listed = 0;
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

  uint32_t T = 0xffffffffu;
  int need_eq = 0;
  if (!take_all && kk > 0) {
    for (int b = lo + tid; b < min(hi, cap); b += kBrThreads) keys[b] = score_key(__ldg(sc + b));
    uint32_t prefix = 0u, mask = 0u;
    int remaining = kk;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int t = lane; t < 256; t += 32) hist[warp][t] = 0;
      __syncthreads();
      for (int b = lo + tid; b < hi; b += kBrThreads) {
        const uint32_t key = key_at(b);
        if ((key & mask) == prefix) atomicAdd(&hist[warp][(key >> shift) & 255u], 1);
      }
      __syncthreads();
      // warp 0: the digit where the count from the top reaches `remaining`;
      // lane l owns digits 8 (31 - l) .. 8 (31 - l) + 7
      if (tid < 256) {
        int t = 0;
#pragma unroll
        for (int w = 0; w < kBrWarps; ++w) t += hist[w][tid];
        hist[0][tid] = t;
      }
      __syncthreads();
      if (warp == 0) {
        const int b0 = 8 * (31 - lane);
        int local = 0;
#pragma unroll
        for (int t = 0; t < 8; ++t) local += hist[0][b0 + t];
        int incl = local;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        int cum = incl - local;
        if (cum < remaining && incl >= remaining) {
          for (int t = 7; t >= 0; --t) {
            const int c = hist[0][b0 + t];
            if (cum + c >= remaining) {
              state[0] = b0 + t;
              state[1] = remaining - cum;
              break;
            }
            cum += c;
          }
        }
      }
      __syncthreads();
      prefix |= (uint32_t)state[0] << shift;
      remaining = state[1];
      mask |= 255u << shift;
    }
    T = prefix;
    need_eq = remaining;
  }

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
  cudaError_t e = cudaFuncSetAttribute(block_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBrCap * 4);
  if (e != cudaSuccess) return e;
  block_rows_kernel<<<dim3(p.Hkv, p.S), kBrThreads, (size_t)cap * 4, st>>>(p, cap);
  return cudaGetLastError();
}

}  // namespace far
