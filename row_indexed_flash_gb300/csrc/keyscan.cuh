// Products of a few query vectors with many keys, reduced per key: the common
// form of the accumulated attention weight (weights.cu) and the block scores
// (blocks.cu).  Keys lie in the M dimension of a tcgen05.mma tile, the query
// vectors of one KV head in N, so that each key's row of products is one
// tensor-memory lane and its reduction over the queries stays in one thread.
#pragma once

#include "fa_internal.cuh"

namespace far {

struct KeyScanParams {
  const void* q;
  const void* k[2];          // weights: {K, -}; scores: {kmax, kmin}
  const uint16_t* k_scale;   // quantised pools (weights)
  const int32_t* rows;       // weights: kv_rows [S, L]; scores: page table [n_seq, L]
  const int32_t* len;        // weights: kv_len [S] or NULL; scores: seq_len [S]
  const int32_t* slice_seq;  // scores: table row of a slice, or NULL
  const float* lse;          // weights
  float* out;                // [S, Hkv, L]: acc or score
  long long R;               // pool rows (weights) or pool pages (scores)
  int S, Nq, Hq, Hkv, L, G, NV, n_seq;   // NV = Nq * G query vectors per KV head
  int q_bf16, causal;
  float c;                   // weights: scale * log2(e)
  float decay;
  unsigned int* err;
  unsigned long long wait_ns;
};

bool keyscan_supported(int D, int G);   // weights: the head dims and groups taken
cudaError_t keyscan_weights(const KeyScanParams& p, int D, int kind, cudaStream_t st);
cudaError_t keyscan_scores(const KeyScanParams& p, int D, cudaStream_t st);

}  // namespace far
