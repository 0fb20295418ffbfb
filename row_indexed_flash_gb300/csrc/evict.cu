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
// shared memory, two or three histograms over the keys' range find the k-th
// largest with the CTAs' histograms added through distributed shared memory,
// and one ordered pass writes the results after the CTAs have exchanged their
// counts.  No scratch in global memory is needed.
//
// Keys beyond the first 40,960 of a CTA's positions do not fit beside and are
// formed from global memory again in every pass: lists longer than 16 times that,
// and, as the SMs are shared out, than twice that from 39 slices on and than
// that from 77.
//
// Bound by latency: each of the five or six exchanges in a cluster costs about
// as much as reading the CTA's totals.  Measured: two slices of 1,000 entries
// 10 us, four of 99,936 entries and 8 KV heads (18 MB) 28 us.
#include <cooperative_groups.h>

#include <atomic>

#include "evict.cuh"
#include "select.cuh"

namespace cg = cooperative_groups;

namespace far {

namespace {

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvPer = 8;            // consecutive positions per thread and step
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

// A position's key from global memory.  Not inlined: the loops that use it for
// the rare positions beyond the on-chip keys stay short (a launch runs its code
// only a few times, so instruction fetches count).
__device__ __noinline__ uint32_t key_from_memory(const float* acc, const int32_t* rows, int pos, int Hkv, int L) {
  return __ldg(rows + pos) >= 0 ? score_key(total_of(acc + pos, Hkv, L)) : 0u;
}

__global__ void __launch_bounds__(kEvThreads, 1) evict_kernel(const EvictParams p, int cap, int vec) {
  extern __shared__ uint32_t keys[];          // [cap] 0: not an entry; later the kept positions
  __shared__ int hist[2][kEvThreads];         // this CTA's histogram, by pass parity
  __shared__ uint32_t ends[2];                // smallest and largest key of this CTA's part of the middle
  __shared__ int warp_sums[kEvWarps + 1];
  __shared__ int all[5];                      // the cluster's sums, or what lies before this CTA
  __shared__ int state[3];
  __shared__ int counts[4];                   // this CTA's entries in the middle, kept, equal to the threshold, live
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31;
  const int s = blockIdx.y;
  const int n = p.kv_len ? min(max(__ldg(p.kv_len + s), 0), p.L) : p.L;
  const int chunk = ((n + C - 1) / C + 31) & ~31;
  const int p0 = min(rank * chunk, n), cnt = min(p0 + chunk, n) - p0;
  const int lo = min(p.sinks, n), hi = max(lo, n - p.recent);   // the middle: [lo, hi)
  const float* acc = p.acc + (size_t)s * p.Hkv * p.L;
  const int32_t* rows = p.kv_rows + (size_t)s * p.L;
  auto make_key = [&](int pos) { return key_from_memory(acc, rows, pos, p.Hkv, p.L); };
  auto key_at = [&](int t) { return t < cap ? keys[t] : make_key(p0 + t); };

  // ---- keys, and the middle's smallest, largest and number
  if (tid == 0) {
    ends[0] = 0xffffffffu;
    ends[1] = 0u;
    counts[0] = 0;
  }
  __syncthreads();
  uint32_t kmin = 0xffffffffu, kmax = 0u;
  int in_middle = 0;
  auto note = [&](int t, uint32_t key) {
    if (t < cap) keys[t] = key;
    if (key != 0u && p0 + t >= lo && p0 + t < hi) {
      kmin = min(kmin, key);
      kmax = max(kmax, key);
      ++in_middle;
    }
  };
  if (vec) {
    // four positions a thread, the loads of up to eight heads in flight
    for (int t = 4 * tid; t < cnt; t += 4 * kEvThreads) {
      if (t + 4 <= cnt) {
        const int4 r = __ldg(reinterpret_cast<const int4*>(rows + p0 + t));
        const float4* a = reinterpret_cast<const float4*>(acc + p0 + t);
        const size_t stride = (size_t)p.L / 4;
        float hi4[4], lo4[4] = {0.f, 0.f, 0.f, 0.f};
        for (int g = 0; g < p.Hkv; g += 8) {
          float4 v[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) v[u] = __ldg(a + (size_t)min(g + u, p.Hkv - 1) * stride);
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            if (g + u >= p.Hkv) break;
            const float x[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (g + u == 0) hi4[e] = x[e];
              else add_exactly(hi4[e], lo4[e], x[e]);
            }
          }
        }
        const int rv[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          note(t + e, rv[e] >= 0 ? score_key(isfinite(hi4[e]) ? hi4[e] + lo4[e] : hi4[e]) : 0u);
      } else {
        for (int e = t; e < cnt; ++e) note(e, make_key(p0 + e));
      }
    }
  } else {
    for (int t = tid; t < cnt; t += kEvThreads) note(t, make_key(p0 + t));
  }
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  in_middle = __reduce_add_sync(0xffffffffu, in_middle);
  if (lane == 0 && in_middle > 0) {
    atomicMin(&ends[0], kmin);
    atomicMax(&ends[1], kmax);
    atomicAdd(&counts[0], in_middle);
  }
  cluster.sync();
  if (tid < 32) {   // lane r reads CTA r
    const bool there = lane < C;
    const uint32_t* e = cluster.map_shared_rank(&ends[0], there ? lane : 0);
    const uint32_t e0 = e[0], e1 = e[1];
    const int c = cluster.map_shared_rank(&counts[0], there ? lane : 0)[0];
    kmin = __reduce_min_sync(0xffffffffu, there ? e0 : 0xffffffffu);
    kmax = __reduce_max_sync(0xffffffffu, there ? e1 : 0u);
    const int sum = __reduce_add_sync(0xffffffffu, there ? c : 0);
    if (lane == 0) {
      all[0] = (int)kmin;
      all[1] = (int)kmax;
      all[2] = sum;
    }
  }
  __syncthreads();
  kmin = (uint32_t)all[0];
  kmax = (uint32_t)all[1];
  const int m = all[2];   // entries of the middle

  // ---- the k-th largest key of the middle's entries
  const bool take_all = m <= p.k, some = !take_all && p.k > 0;
  KeyRange range = key_range(kmin, kmax, p.k);
  for (int pass = 0; some && !range.done; ++pass) {
    int* mine = hist[pass & 1];
    mine[tid] = 0;
    __syncthreads();
    const int shift = range_shift<kEvThreads>(range);
    for (int t = tid; t < cnt; t += kEvThreads) {
      const int pos = p0 + t;
      const uint32_t key = key_at(t);
      if (key != 0u && pos >= lo && pos < hi && in_range(range, key)) atomicAdd(&mine[(key - range.base) >> shift], 1);
    }
    // A CTA clears this histogram again two passes on, after a cluster barrier
    // that every reader of this pass has reached
    cluster.sync();
    int c = 0;
#pragma unroll
    for (int r = 0; r < kEvMaxCluster; ++r)
      if (r < C) c += cluster.map_shared_rank(mine, r)[kEvThreads - 1 - tid];
    range_pick<kEvThreads>(range, c, warp_sums, state);
    __syncthreads();   // state may be written again
  }
  const uint32_t T = range.T;
  const int need_eq = range.need_eq;
  // 0: dropped, 1: kept, 2: kept if among the first need_eq equal ones
  auto verdict = [&](int pos, uint32_t key) {
    const bool forced = take_all | (pos < lo) | (pos >= hi);
    const int by_key = key > T ? 1 : key == T ? 2 : 0;
    return key == 0u ? 0 : forced ? 1 : by_key;
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
  if (tid < 4) warp_sums[tid] = 0;
  __syncthreads();
  c_keep = __reduce_add_sync(0xffffffffu, c_keep);
  c_eq = __reduce_add_sync(0xffffffffu, c_eq);
  c_live = __reduce_add_sync(0xffffffffu, c_live);
  if (lane == 0) {
    atomicAdd(&warp_sums[0], c_keep);
    atomicAdd(&warp_sums[1], c_eq);
    atomicAdd(&warp_sums[2], c_live);
  }
  __syncthreads();
  if (tid < 3) counts[1 + tid] = warp_sums[tid];   // counts[0] may still be read by other CTAs
  cluster.sync();
  if (tid < 32) {
    const bool there = lane < C, before = lane < rank;
    const int* c = cluster.map_shared_rank(&counts[0], there ? lane : 0);
    const int a = c[1], e = c[2], l = c[3];
    // sums over the CTAs before this one, and over all
    const int v[6] = {__reduce_add_sync(0xffffffffu, before ? a : 0), __reduce_add_sync(0xffffffffu, before ? e : 0),
                      __reduce_add_sync(0xffffffffu, before ? l : 0), __reduce_add_sync(0xffffffffu, there ? a : 0),
                      __reduce_add_sync(0xffffffffu, there ? e : 0), __reduce_add_sync(0xffffffffu, there ? l : 0)};
    if (lane == 0) {
      const int kept_before = v[0] + min(v[1], need_eq);
      all[0] = kept_before;
      all[1] = v[1];
      all[2] = v[2] - kept_before;
      all[3] = v[3] + min(v[4], need_eq);
      all[4] = v[5];
    }
  }
  __syncthreads();
  int out_at = all[0], eq_seen = all[1], drop_at = all[2];
  const int n_keep = all[3], n_live = all[4];

  // ---- ordered pass
  int32_t* rows_out = p.rows_out + (size_t)s * p.out_len;
  int32_t* kept = p.kept ? p.kept + (size_t)s * p.out_len : nullptr;
  int32_t* freed = p.freed ? p.freed + (size_t)s * p.L : nullptr;
  float* acc_out = p.acc_out + (size_t)s * p.Hkv * p.out_len;
  const int out_first = out_at;
  for (int base = 0; base < cnt; base += kEvThreads * kEvPer) {
    const int t0 = base + tid * kEvPer;
    int v[kEvPer], row[kEvPer];
    unsigned live = 0u;
    int n_eq = 0;
    // the rows that may be freed, loaded while the counts are formed
#pragma unroll
    for (int u = 0; u < kEvPer; ++u) row[u] = freed && t0 + u < cnt ? __ldg(rows + p0 + t0 + u) : -1;
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
        // Noted for the copy below, in a key's place: a kept entry's number is
        // no larger than its position, and every key up to this step's end
        // has been read.
        if (at - out_first < cap) {
          keys[at - out_first] = (uint32_t)pos;
        } else {
          rows_out[at] = __ldg(rows + pos);
          if (kept) kept[at] = pos;
          for (int g = 0; g < p.Hkv; ++g) acc_out[(size_t)g * p.out_len + at] = __ldg(acc + (size_t)g * p.L + pos);
        }
        ++at;
      } else if ((live >> u) & 1u) {
        if (freed) freed[dat] = row[u];
        ++dat;
      }
    }
    out_at += total & 0xffff;
    drop_at += total >> 16;
    eq_seen += eq_total;
  }
  __syncthreads();
  // ---- the kept entries: neighbouring threads, neighbouring outputs
  const int mine_kept = min(out_at - out_first, cap);
  for (int i = tid; i < mine_kept; i += kEvThreads) {
    const int pos = (int)keys[i];
    rows_out[out_first + i] = __ldg(rows + pos);
    if (kept) kept[out_first + i] = pos;
    for (int g = 0; g < p.Hkv; g += 8) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = __ldg(acc + (size_t)min(g + u, p.Hkv - 1) * p.L + pos);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (g + u < p.Hkv) acc_out[(size_t)(g + u) * p.out_len + out_first + i] = v[u];
    }
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

cudaError_t evict_launch(const EvictParams& p, cudaStream_t st) {
  // CTAs per slice: enough for about 2048 positions each, no more than the
  // SMs there are for all slices
  int C = 1;
  while (C < kEvMaxCluster && p.L > C * 2048 && (long long)p.S * C * 2 <= sm_count()) C *= 2;
  const int chunk = ((p.L + C - 1) / C + 31) & ~31;
  const int cap = chunk < kEvCap ? chunk : kEvCap;
  const cudaError_t e = once_per_device<0>([] {
    cudaError_t x = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvCap * 4);
    return x == cudaSuccess ? cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) : x;
  });
  if (e != cudaSuccess) return e;
  // 16-byte loads of the totals and rows
  const int vec = p.L % 4 == 0 && reinterpret_cast<uintptr_t>(p.acc) % 16 == 0 && reinterpret_cast<uintptr_t>(p.kv_rows) % 16 == 0;
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
  return cudaLaunchKernelEx(&cfg, evict_kernel, p, cap, vec);
}

}  // namespace far
