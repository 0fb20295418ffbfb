// Launch parameters of the eviction (evict.cu).
#pragma once

#include "fa_internal.cuh"

namespace far {

struct EvictParams {
  const float* acc;
  const int32_t* kv_rows;
  const int32_t* kv_len;
  float* acc_out;
  int32_t* rows_out;
  int32_t* len_out;
  int32_t* kept;    // NULL: not wanted
  int32_t* freed;   // NULL: not wanted
  int S, Hkv, L, sinks, recent, k, out_len;
};
cudaError_t evict_launch(const EvictParams& p, cudaStream_t st);

}  // namespace far
