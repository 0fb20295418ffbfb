// Eviction from a row list by accumulated attention weight.
//
// Per slice, with total[j] = sum over KV heads of acc[s, g, j]: the entries
// kept are the first `sinks` and last `recent` list positions and the k
// positions between them with the largest totals (ties to the smaller
// position, NaN below every number); padding entries are never kept.  The
// list, the positions and every head's totals of the kept entries are written
// compacted in position order, and the rows of the others are reported.
//
// One thread-block cluster per slice, each CTA owning a run of positions: one
// pass over the totals leaves an order-preserving 32-bit key per position in
// shared memory, a radix selection (four 8-bit digits) finds the k-th largest
// key with the CTAs' histograms added through distributed shared memory, and
// one ordered pass writes the results after the CTAs have exchanged their
// counts.  Nothing but the kernel's own inputs is re-read, and no scratch in
// global memory is needed.
#include <cooperative_groups.h>

#include <atomic>

#include "evict.cuh"
#include "select.cuh"

namespace cg = cooperative_groups;

namespace far {

namespace {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvPer = 4;            // consecutive positions per thread and step
constexpr int kEvCap = 40960;        // positions per CTA whose keys are kept in shared memory
constexpr int kEvMaxCluster = 16;

// Two fp32 terms that hold a sum to about 48 bits: a + b exactly as hi + lo.
__device__ __forceinline__ void add_exactly(float& hi, float& lo, float b) {
  const float s = hi + b, t = s - hi;
  lo += (hi - (s - t)) + (b - t);
  hi = s;
}

// The entry's total over the KV heads, rounded once to fp32.  (An infinite or
// NaN sum keeps its value: its error term means nothing.)
__device__ __forceinline__ float total_of(const float* a, int Hkv, size_t stride) {
  float hi = __ldg(a), lo = 0.f;
  for (int g = 1; g < Hkv; ++g) add_exactly(hi, lo, __ldg(a + g * stride));
  return isfinite(hi) ? hi + lo : hi;
}

__global__ void __launch_bounds__(kEvThreads, 1) evict_kernel(const EvictParams p, int cap) {
  extern __shared__ uint32_t keys[];          // [cap] 0: not an entry
  __shared__ int hist[kEvWarps][256];
  __shared__ int digits[2][256];              // this CTA's histogram, by pass parity
  __shared__ int warp_sums[kEvWarps];
  __shared__ int state[2];
  __shared__ int counts[4];                   // this CTA's kept, equal to the threshold, live
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = blockIdx.y;
  const int n = p.kv_len ? min(max(__ldg(p.kv_len + s), 0), p.L) : p.L;
  const int chunk = ((n + C - 1) / C + 31) & ~31;
  const int p0 = min(rank * chunk, n), cnt = min(p0 + chunk, n) - p0;
  const int lo = min(p.sinks, n), hi = max(lo, n - p.recent);   // the middle: [lo, hi)
  const float* acc = p.acc + (size_t)s * p.Hkv * p.L;
  const int32_t* rows = p.kv_rows + (size_t)s * p.L;
  auto make_key = [&](int pos) {
    return __ldg(rows + pos) >= 0 ? score_key(total_of(acc + pos, p.Hkv, p.L)) : 0u;
  };
  auto key_at = [&](int t) { return t < cap ? keys[t] : make_key(p0 + t); };

  for (int t = tid; t < min(cnt, cap); t += kEvThreads) keys[t] = make_key(p0 + t);

  // ---- the k-th largest key of the middle's entries
  uint32_t prefix = 0u, mask = 0u;
  int remaining = p.k;
  bool take_all = false;
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int t = lane; t < 256; t += 32) hist[warp][t] = 0;
    __syncthreads();
    for (int t = tid; t < cnt; t += kEvThreads) {
      const int pos = p0 + t;
      const uint32_t key = key_at(t);
      if (key != 0u && pos >= lo && pos < hi && (key & mask) == prefix) atomicAdd(&hist[warp][(key >> shift) & 255u], 1);
    }
    __syncthreads();
    if (tid < 256) {
      int t = 0;
#pragma unroll
      for (int w = 0; w < kEvWarps; ++w) t += hist[w][tid];
      digits[pass & 1][tid] = t;
    }
    cluster.sync();
    // a CTA writes digits[parity] again two passes on, after a cluster barrier
    // that every reader of this pass has reached
    if (tid < 256) {
      int t = 0;
      for (int r = 0; r < C; ++r) t += cluster.map_shared_rank(&digits[pass & 1][0], r)[tid];
      hist[0][tid] = t;
    }
    __syncthreads();
    if (warp == 0) {
      // lane l owns digits 8 (31 - l) .. 8 (31 - l) + 7
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
      const int all = __shfl_sync(0xffffffffu, incl, 31);
      int cum = incl - local;
      if (pass == 0 && all <= remaining) {   // every entry of the middle is kept
        if (lane == 0) state[0] = -1;
      } else if (cum < remaining && incl >= remaining) {
        for (int t = 7; t >= 0; --t) {
          const int c = hist[0][b0 + t];
          if (cum + c >= remaining) {
            state[0] = b0 + t;
            state[1] = remaining - cum;
            break;
          }
          cum += c;
        }
      } else if (remaining == 0 && lane == 0) {
        state[0] = -2;
      }
    }
    __syncthreads();
    const int digit = state[0];
    __syncthreads();
    if (digit < 0) {
      take_all = digit == -1;
      break;
    }
    prefix |= (uint32_t)digit << shift;
    remaining = state[1];
    mask |= 255u << shift;
    if (pass == 3) break;
  }
  const bool some = mask == 0xffffffffu;
  const uint32_t T = some ? prefix : 0xffffffffu;
  const int need_eq = some ? remaining : 0;
  // 0: dropped, 1: kept, 2: kept if among the first need_eq equal ones
  auto verdict = [&](int pos, uint32_t key) {
    if (key == 0u) return 0;
    if (pos < lo || pos >= hi || take_all) return 1;
    if (!some) return 0;
    return key > T ? 1 : key == T ? 2 : 0;
  };

  // ---- this CTA's counts, exchanged
  int c_keep = 0, c_eq = 0, c_live = 0;
  for (int t = tid; t < cnt; t += kEvThreads) {
    const uint32_t key = key_at(t);
    const int v = verdict(p0 + t, key);
    c_keep += v == 1;
    c_eq += v == 2;
    c_live += key != 0u;
  }
  if (tid < 4) counts[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    c_keep += __shfl_xor_sync(0xffffffffu, c_keep, o);
    c_eq += __shfl_xor_sync(0xffffffffu, c_eq, o);
    c_live += __shfl_xor_sync(0xffffffffu, c_live, o);
  }
  if (lane == 0) {
    atomicAdd(&counts[0], c_keep);
    atomicAdd(&counts[1], c_eq);
    atomicAdd(&counts[2], c_live);
  }
  cluster.sync();
  int out_at = 0, eq_seen = 0, live_before = 0, n_keep = 0, n_eq_all = 0, n_live = 0;
  for (int r = 0; r < C; ++r) {
    const int* c = cluster.map_shared_rank(&counts[0], r);
    const int a = c[0], e = c[1], l = c[2];
    if (r < rank) {
      out_at += a;
      eq_seen += e;
      live_before += l;
    }
    n_keep += a;
    n_eq_all += e;
    n_live += l;
  }
  out_at += min(eq_seen, need_eq);
  n_keep += min(n_eq_all, need_eq);
  int drop_at = live_before - out_at;

  // ---- ordered pass
  int32_t* rows_out = p.rows_out + (size_t)s * p.out_len;
  int32_t* kept = p.kept ? p.kept + (size_t)s * p.out_len : nullptr;
  int32_t* freed = p.freed ? p.freed + (size_t)s * p.L : nullptr;
  float* acc_out = p.acc_out + (size_t)s * p.Hkv * p.out_len;
  for (int base = 0; base < cnt; base += kEvThreads * kEvPer) {
    const int t0 = base + tid * kEvPer;
    int v[kEvPer];
    unsigned live = 0u;
    int n_eq = 0;
#pragma unroll
    for (int u = 0; u < kEvPer; ++u) {
      const uint32_t key = t0 + u < cnt ? key_at(t0 + u) : 0u;
      v[u] = verdict(p0 + t0 + u, key);
      live |= (key != 0u ? 1u : 0u) << u;
      n_eq += v[u] == 2;
    }
    int eq_total = 0;
    int eq = eq_seen + block_scan<kEvThreads>(n_eq, warp_sums, &eq_total);
    unsigned sel = 0u;
#pragma unroll
    for (int u = 0; u < kEvPer; ++u) {
      bool on = v[u] == 1;
      if (v[u] == 2) on = eq++ < need_eq;
      sel |= (on ? 1u : 0u) << u;
    }
    // kept and dropped counts of a step fit 16 bits each
    int total = 0;
    const int before = block_scan<kEvThreads>(__popc(sel) | (__popc(live & ~sel) << 16), warp_sums, &total);
    int at = out_at + (before & 0xffff), dat = drop_at + (before >> 16);
#pragma unroll
    for (int u = 0; u < kEvPer; ++u) {
      const int pos = p0 + t0 + u;
      if ((sel >> u) & 1u) {
        rows_out[at] = __ldg(rows + pos);
        if (kept) kept[at] = pos;
        for (int g = 0; g < p.Hkv; ++g) acc_out[(size_t)g * p.out_len + at] = __ldg(acc + (size_t)g * p.L + pos);
        ++at;
      } else if ((live >> u) & 1u) {
        if (freed) freed[dat] = __ldg(rows + pos);
        ++dat;
      }
    }
    out_at += total & 0xffff;
    drop_at += total >> 16;
    eq_seen += eq_total;
  }
  // ---- padding, spread over the cluster
  const int step = C * kEvThreads, me = rank * kEvThreads + tid;
  for (int j = n_keep + me; j < p.out_len; j += step) {
    rows_out[j] = -1;
    if (kept) kept[j] = -1;
    for (int g = 0; g < p.Hkv; ++g) acc_out[(size_t)g * p.out_len + j] = 0.f;
  }
  if (freed)
    for (int j = n_live - n_keep + me; j < p.L; j += step) freed[j] = -1;
  if (me == 0) p.len_out[s] = n_keep;
  cluster.sync();   // no CTA leaves while another may still read its shared memory
}

}  // namespace

cudaError_t evict_launch(const EvictParams& p, int sm_count, cudaStream_t st) {
  // CTAs per slice: enough for about 2048 positions each, no more than the
  // SMs there are for all slices
  int C = 1;
  while (C < kEvMaxCluster && p.L > C * 2048 && (long long)p.S * C * 2 <= sm_count) C *= 2;
  const int chunk = ((p.L + C - 1) / C + 31) & ~31;
  const int cap = chunk < kEvCap ? chunk : kEvCap;
  cudaError_t e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvCap * 4);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C, p.S);
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = (size_t)cap * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_kernel, p, cap);
}

}  // namespace far
