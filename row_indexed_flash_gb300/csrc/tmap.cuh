// Host side: encoding of TMA tensor maps through the CUDA driver API entry point, with
// a cache so that repeated calls on the same tensors (a decode step per
// token) skip the encode.  Shared by the kernels' launch code.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <string.h>

#include <mutex>

namespace far {

inline PFN_cuTensorMapEncodeTiled_v12000 tmap_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// The encodings of the last tensors, by everything an encoding depends on.  A
// prefill call takes five maps and a decode call two, and every layer of a
// model has a pool of its own: sets of eight, found by a hash, hold those of 100
// layers and more.  (The 32 that were searched in a row held six prefill layers.)
struct TmapKey {
  const void* base;
  cuuint64_t dims[3], strides[2];
  cuuint32_t box[3];
  int dt, sw, dev;
};
class TmapCache {
 public:
  bool find(const TmapKey& key, CUtensorMap* m) {
    std::lock_guard<std::mutex> lock(mu_);
    const Set& s = set_[index(key)];
    for (int i = 0; i < kWays; ++i)
      if (s.used[i] && memcmp(&s.key[i], &key, sizeof(key)) == 0) {
        *m = s.map[i];
        return true;
      }
    return false;
  }
  void put(const TmapKey& key, const CUtensorMap& m) {
    std::lock_guard<std::mutex> lock(mu_);
    Set& s = set_[index(key)];
    const int i = s.next;
    s.key[i] = key;
    s.map[i] = m;
    s.used[i] = true;
    s.next = (i + 1) % kWays;
  }

 private:
  static constexpr int kSets = 128, kWays = 8;
  struct Set {
    CUtensorMap map[kWays];
    TmapKey key[kWays];
    bool used[kWays];
    int next;
  };
  static int index(const TmapKey& key) {
    static_assert(sizeof(TmapKey) % 8 == 0, "whole words");
    unsigned long long w[sizeof(TmapKey) / 8], h = 0;
    memcpy(w, &key, sizeof(key));
    for (unsigned long long x : w) {
      h = (h ^ x) * 0x9e3779b97f4a7c15ull;   // an odd multiplier: 2^64 over the golden ratio
      h ^= h >> 32;
    }
    return (int)(h % kSets);
  }
  Set set_[kSets] = {};
  std::mutex mu_;
};

// A 3-D tiled map (unit element strides, no interleave, 256-byte L2
// promotion, zero fill).
inline bool tmap_encode_3d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, const cuuint64_t (&dims)[3],
                           const cuuint64_t (&strides)[2], const cuuint32_t (&box)[3], CUtensorMapSwizzle sw) {
  static TmapCache cache;
  TmapKey key;
  memset(&key, 0, sizeof(key));   // padding bytes take part in the comparison
  key.base = base;
  for (int i = 0; i < 3; ++i) key.dims[i] = dims[i], key.box[i] = box[i];
  for (int i = 0; i < 2; ++i) key.strides[i] = strides[i];
  key.dt = (int)dt;
  key.sw = (int)sw;
  if (cudaGetDevice(&key.dev) != cudaSuccess) key.dev = -1;
  if (cache.find(key, m)) return true;
  auto enc = tmap_encode_fn();
  if (!enc) return false;
  const cuuint32_t es[3] = {1, 1, 1};
  if (enc(m, dt, 3, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  cache.put(key, *m);
  return true;
}

}  // namespace far
