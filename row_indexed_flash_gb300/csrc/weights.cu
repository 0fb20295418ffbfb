// Attention weight received by every listed cache entry, accumulated.
//
// For slice s, KV head g and list position j,
//   acc[s, g, j] = decay * acc[s, g, j]
//                + sum over queries i and heads h of group g of exp(scale * <q[s,i,h], K[row_j, g]> + mask - lse[s,i,h])
// where lse is what the attention call over the same lists returned, so each
// term is exactly the softmax weight that call gave the entry.  A query with
// no visible entry (lse = -inf) adds nothing.  Each (s, g, j) is owned by one
// thread and its terms are added in one fixed order: no atomics, the same bits
// every time.
//
// This file holds the CUDA-core kernel, for what the tensor-core kernels
// (keyscan.cu) do not take: dense masks, head dims other than 64, 128 and 256,
// unaligned Q, very wide groups (4 x 16,384 rows, D 128, four query vectors:
// 198 us here, 30 us there).  A CTA stages 128 listed keys as fp32 (codes times scale: exact) in shared
// memory, one thread per key forms the logits of eight query vectors at a time
// (broadcast reads of the staged queries) and adds their weights.  Rows are
// padded by one word, so the 32 keys of a warp lie on 32 banks.
#include <string.h>

#include "fa_internal.cuh"
#include "keyscan.cuh"
#include "kvread.cuh"
#include "weights.cuh"

namespace far {

namespace {

constexpr int kWKeys = 128;   // keys per CTA = threads
constexpr int kWVec = 8;      // query vectors per pass

template <int KIND>
__global__ void __launch_bounds__(kWKeys) weights_generic_kernel(const WeightsParams p) {
  extern __shared__ float wsm[];
  const int D = p.D, KS = D + 1;
  float* ks = wsm;                         // [kWKeys][D + 1]
  float* qs = wsm + kWKeys * KS;           // [kWVec][D]
  float* ls = qs + kWVec * D;              // [kWVec] log-sum-exp
  const int tid = threadIdx.x;
  const int s = blockIdx.z, g = blockIdx.y, j0 = blockIdx.x * kWKeys;
  const int n_s = p.kv_len ? min(max(__ldg(p.kv_len + s), 0), p.L) : p.L;
  if (j0 >= n_s) return;
  const int j = j0 + tid;
  int row = j < n_s ? __ldg(p.kv_rows + (size_t)s * p.L + j) : -1;
  if ((long long)row >= p.R) row = -1;

  // stage the keys: 16-byte chunks of one row by consecutive threads
  const int cpr = kv_row_bytes<KIND>(D) / 16;
  __shared__ int rows_s[kWKeys];
  rows_s[tid] = row;
  __syncthreads();
  for (int f = tid; f < kWKeys * cpr; f += kWKeys) {
    const int e = f / cpr, c = f % cpr, r = rows_s[e];
    float x[KvChunk<KIND>::N];
    kv_chunk<KIND>(p.k, p.k_scale, r, g, p.Hkv, D, c, x);
#pragma unroll
    for (int t = 0; t < KvChunk<KIND>::N; ++t) ks[e * KS + c * KvChunk<KIND>::N + t] = x[t];
  }

  const int nv = p.Nq * p.G;
  float total = 0.f;
  for (int v0 = 0; v0 < nv; v0 += kWVec) {
    __syncthreads();
    const int m = min(kWVec, nv - v0);
    for (int f = tid; f < m * D; f += kWKeys) {
      const int v = v0 + f / D, d = f % D;
      const size_t qi = (((size_t)s * p.Nq + v / p.G) * p.Hq + g * p.G + v % p.G);
      const uint16_t u = __ldg(static_cast<const uint16_t*>(p.q) + qi * D + d);
      qs[f] = p.q_bf16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
    }
    if (tid < m) {
      const int v = v0 + tid;
      ls[tid] = __ldg(p.lse + ((size_t)s * p.Nq + v / p.G) * p.Hq + g * p.G + v % p.G);
    }
    __syncthreads();
    if (row < 0) continue;
    float dot[kWVec];
#pragma unroll
    for (int t = 0; t < kWVec; ++t) dot[t] = 0.f;
    for (int d = 0; d < D; ++d) {
      const float k = ks[tid * KS + d];
#pragma unroll
      for (int t = 0; t < kWVec; ++t) dot[t] = fmaf(qs[t * D + d], k, dot[t]);
    }
    float part = 0.f;
#pragma unroll
    for (int t = 0; t < kWVec; ++t) {
      if (t >= m) break;
      const int i = (v0 + t) / p.G;
      if (p.mask_kind == FA_MASK_CAUSAL && j > n_s - p.Nq + i) continue;
      const float l = ls[t];
      if (l == __int_as_float(0xff800000)) continue;
      float x = dot[t] * p.scale;
      if (p.mask_kind == FA_MASK_DENSE) {
        const float mv = __ldg(p.mask + ((size_t)s * p.Nq + i) * p.L + j);
        if (mv == __int_as_float(0xff800000)) continue;
        x += mv;
      }
      part += fast_ex2((x - l) * kLog2e);
    }
    total += part;
  }
  if (j < n_s) {
    float* a = p.acc + ((size_t)s * p.Hkv + g) * p.L + j;
    *a = p.decay == 0.f ? total : fmaf(p.decay, *a, total);
  }
}

constexpr int kWMaxD = 256;
constexpr size_t weights_smem(int D) { return ((size_t)kWKeys * (D + 1) + kWVec * D + kWVec) * sizeof(float); }

template <int KIND>
cudaError_t weights_generic(const WeightsParams& p, cudaStream_t st) {
  if (p.D > kWMaxD) return cudaErrorInvalidValue;
  const size_t smem = weights_smem(p.D);
  // the limit of the largest call, once: the attribute is the device's, and
  // another thread's call may lie between its setting and this launch
  const cudaError_t e = once_per_device<5>([] {
    return cudaFuncSetAttribute(weights_generic_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)weights_smem(kWMaxD));
  });
  if (e != cudaSuccess) return e;
  const dim3 grid((p.L + kWKeys - 1) / kWKeys, p.Hkv, p.S);
  weights_generic_kernel<KIND><<<grid, kWKeys, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t weights_launch(const WeightsParams& p, cudaStream_t st) {
  const int nv = p.Nq * p.G;
  if (p.mask_kind != FA_MASK_DENSE && reinterpret_cast<uintptr_t>(p.q) % 16 == 0 && keyscan_supported(p.D, p.G)) {
    KeyScanParams k;
    memset(&k, 0, sizeof(k));
    k.q = p.q;
    k.k[0] = p.k;
    k.k_scale = p.k_scale;
    k.rows = p.kv_rows;
    k.len = p.kv_len;
    k.lse = p.lse;
    k.out = p.acc;
    k.R = p.R;
    k.S = p.S;
    k.Nq = p.Nq;
    k.Hq = p.Hq;
    k.Hkv = p.Hkv;
    k.L = p.L;
    k.G = p.G;
    k.NV = nv;
    k.n_seq = p.S;
    k.q_bf16 = p.q_bf16;
    k.causal = p.mask_kind == FA_MASK_CAUSAL;
    k.c = p.scale * kLog2e;
    k.decay = p.decay;
    k.err = p.err;
    k.wait_ns = p.wait_ns;
    return keyscan_weights(k, p.D, p.kind, st);
  }
  switch (p.kind) {
    case KV_BF16: return weights_generic<KV_BF16>(p, st);
    case KV_F16: return weights_generic<KV_F16>(p, st);
    case KV_I8: return weights_generic<KV_I8>(p, st);
    case KV_I4: return weights_generic<KV_I4>(p, st);
    case KV_F8: return weights_generic<KV_F8>(p, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace far
