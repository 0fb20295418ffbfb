// Launch parameters of the accumulated attention weight (weights.cu).
#pragma once

#include "fa_internal.cuh"

namespace far {

struct WeightsParams {
  const void* q;
  const void* k;
  const uint16_t* k_scale;
  const int32_t* kv_rows;
  const int32_t* kv_len;
  const float* mask;
  const float* lse;
  float* acc;
  long long R;
  int S, Nq, Hq, Hkv, L, G, D;
  int kind;            // KvKind of the pool
  int q_bf16;
  int mask_kind;       // fa_mask_kind
  float scale, decay;
  unsigned int* err;   // the workspace status word
  unsigned long long wait_ns;
};

cudaError_t weights_launch(const WeightsParams& p, cudaStream_t st);

}  // namespace far
