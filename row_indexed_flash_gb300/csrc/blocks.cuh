// Launch parameters of the block operators (blocks.cu).
#pragma once

#include "fa_internal.cuh"

namespace far {

struct BoundsParams {
  const void* k;
  const uint16_t* k_scale;
  const int32_t* pages;
  const int32_t* fill;   // NULL: full pages
  void* kmin;
  void* kmax;
  long long n_pool_pages;
  int n_pages, Hkv, D, kind;
  int out_bf16;
};
cudaError_t bounds_launch(const BoundsParams& p, cudaStream_t st);

struct ScoresParams {
  const void* q;
  const void* kmin;
  const void* kmax;
  const int32_t* page_table;
  const int32_t* seq_len;
  const int32_t* slice_seq;   // NULL: slice s uses table row s
  float* score;
  long long n_pool_pages;
  int S, Nq, Hq, Hkv, G, D, max_pages, n_seq;
  int q_bf16;
  unsigned int* err;
  unsigned long long wait_ns;
};
cudaError_t scores_launch(const ScoresParams& p, cudaStream_t st);

struct BlockRowsParams {
  const float* score;
  const int32_t* page_table;
  const int32_t* seq_len;
  const int32_t* slice_seq;
  int32_t* kv_rows;
  int32_t* kv_len;
  int S, Hkv, max_pages, n_seq, sinks, recent, k, list_len;
};
cudaError_t block_rows_launch(const BlockRowsParams& p, cudaStream_t st);

}  // namespace far
