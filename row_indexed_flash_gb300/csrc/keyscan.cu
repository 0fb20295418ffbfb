// Few query vectors against many keys on the 5th-generation tensor cores.
//
//   weights  acc[s, g, j] = decay * acc + sum_v exp2(c * <q_v, K[row_j, g]> - lse2_v)
//   scores   score[s, g, b] = max_v <max(q_v, 0), kmax[page_b, g]> + <min(q_v, 0), kmin[page_b, g]>
//            (an infinite bound counts only for the signs that use it: score_by_definition)
//
// Bound by the bytes of the keys: each is read once.  The keys of a tile are
// the 128 rows of the MMA's M dimension and the few query vectors of the KV
// head its N columns, so a key's products lie in one tensor-memory lane
// and one thread reduces them in registers, in a fixed order, with nothing
// exchanged between threads and one fp32 written per key.
//
// One CTA per SM walks an even share of all (slice, KV head, tile) triples,
// whatever the slices' lengths: every CTA adds up the tile counts itself and
// finds its first triple (list lengths are on the device).  Warps:
//   0-7    reduction: two warpgroups on alternate tiles; thread t owns key t of
//          the tile: tensor-memory loads of its row, the reduction, the update
//          of the output
//   8      MMA issue; allocates tensor memory
//   9      queries of the next (slice, KV head), into one of two buffers: its
//          rows and, for weights, lse in log2 units and the causal limits
//   10 on  keys: two groups of four warps (eight for codes) on alternate tiles
//          (one group's instructions per tile take longer than the tile's share
//          of HBM time), half of them for each 64-row half; cp.async of the
//          listed rows into the 128-byte-swizzled layout, or one TMA tile load
//          per 64 columns where the half is one contiguous pool run.  The
//          copies arrive on the stage's barrier by themselves.
// Scores take two stages per tile (kmax with max(q, 0), then kmin with
// min(q, 0)), accumulated by the tensor core.  Codes of quantised pools are
// copied to a ring in shared memory, widened exactly to Q's type by the lanes
// that copied them, and the row's scale multiplies the product afterwards.
// Every wait is bounded in time and reported through the workspace's status word.
//
// Measured, 4 slices x 16,384 listed rows of a shuffled pool, 8 KV heads, D 128,
// four query vectors each (136 MB of keys and totals): 30 us, 4.6 TB/s; another
// 16,384 rows per slice add 22 us, 6.3 TB/s (0.93 of the copy rate), so what
// keeps the short call from it is about 6 us of start and end (a call of one
// tile per CTA takes that).  INT8 33 us, INT4 32 us, E4M3 36 us: not the bytes
// (INT4 has half of INT8's) nor widening as such (the quantised decode, where
// some warps only copy and others only widen, takes in bytes at twice INT8's
// rate here) but each key warp's own chain of copy, widen and wait for a stage.
// Scores of 32 sequences of 1k to 128k tokens (58 MB of bounds) 22 us.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <string.h>

#include "keyscan.cuh"
#include "kvread.cuh"
#include "tc.cuh"
#include "tmap.cuh"
#include "widen.cuh"

namespace far {

namespace ks {
constexpr int BM = 128;                    // keys per tile
constexpr int NEPI = 8, W_MMA = 8, W_Q = 9, W_KEY = 10;
// Key warps: widening codes takes twice the warps that copies alone do.
template <bool QUANT>
constexpr int kKeyWarps = QUANT ? 16 : 8;
template <bool QUANT>
constexpr int kThreads = (W_KEY + kKeyWarps<QUANT>) * 32;
constexpr int NBUF = 4;                    // accumulators
constexpr int MAXST = 8;                  // stages
constexpr int MAXN = 128;                  // query vectors, at most (see kStreamVec)
constexpr int PRE = 3;                     // own tiles ahead that a key warp loads list entries
// Groups of key warps on alternate tiles: two, but one for the codes of D 256
// (two groups' code rings do not fit beside their operand stage) and for its
// scores (two or fewer stages).  A stage's barrier tells two neighbouring
// phases apart, so with two groups there must be more stages than a tile uses:
// then whoever waits for a stage's last use knows that the use before it is over.
template <int D, int NK, bool QUANT>
constexpr int kGroups = D > 128 && (QUANT || NK == 2) ? 1 : 2;
constexpr int SMEM_MAX = 225 * 1024;
// Query vectors that the streaming form takes; more go to the prompt form.  Four
// slices of 16,384 entries, D 128, bf16, 8 heads: 64 vectors 33 us here and 60
// there, 128 vectors 42 us here and 59 there.  With two D-wide query parts
// (scores), codes or D 256 only 64 vectors leave room for the stages.
template <int D, int NK, bool QUANT>
constexpr int kStreamVec = NK == 1 && !QUANT && D <= 128 ? 128 : 64;
// Accumulators per tile: at D 256 the two products of a score have one each and
// are added in fp32.  The tensor core cuts its running sum off rather than
// rounding it, and the terms of a score mostly have one sign, so 32 steps into
// one accumulator left f16 scores 1.6e-6 low; 16 into each of two leave half that.
template <int D, int NK>
constexpr int kParts = NK == 2 && D == 256 ? 2 : 1;
}  // namespace ks

namespace {

enum { SCAN_WEIGHTS = 0, SCAN_SCORES = 1 };

// Tiles of codes that a group of key warps has in flight beside the one it
// widens: as many as the shared memory beside 64 query vectors and the operand
// stages holds, at most PRE.
template <int D, int KIND>
__host__ __device__ constexpr int ks_ahead() {
  const int code = ks::kGroups<D, 1, true> * ks::BM * kv_row_bytes<KIND>(D);
  const int room = ks::SMEM_MAX - 4096 - 2 * ks::kStreamVec<D, 1, true> * D * 2 - (D <= 128 ? 2 : 1) * ks::BM * D * 2;
  const int n = room / code - 1;
  return n > ks::PRE ? ks::PRE : n;
}

// Shared memory of one instance: sizes that depend on N and the stage counts
// are computed the same way on both sides.
struct KsLayout {
  int N, qb_bytes, nst, tile, ncs, code, off_q, off_k, off_c, off_bar, off_misc, off_l, total;
};

template <int D, int MODE, int KIND>
__host__ __device__ inline KsLayout ks_layout(int nv) {
  constexpr bool QUANT = KIND == KV_I8 || KIND == KV_I4 || KIND == KV_F8;
  KsLayout l;
  l.N = (nv + 15) / 16 * 16;
  const int kd = MODE == SCAN_SCORES ? 2 * D : D;
  l.qb_bytes = l.N * kd * 2;
  l.tile = ks::BM * D * 2;
  l.code = QUANT ? ks::BM * kv_row_bytes<KIND>(D) : 0;
  l.off_q = 0;
  l.off_k = (2 * l.qb_bytes + 1023) / 1024 * 1024;
  const int room = ks::SMEM_MAX - 1024 - l.off_k - 3 * 1024;
  if (QUANT) {
    // the code ring, operand stages with what is left (two at least; one for D 256)
    l.ncs = ks::kGroups<D, 1, true> * (ks_ahead<D, KIND>() + 1);
    l.nst = (room - l.ncs * l.code) / l.tile;
    l.nst = l.nst > ks::MAXST ? ks::MAXST : l.nst;
  } else {
    l.nst = room / l.tile;
    l.nst = l.nst > ks::MAXST ? ks::MAXST : l.nst;
    l.ncs = 0;
  }
  l.off_c = l.off_k + l.nst * l.tile;
  l.off_bar = l.off_c + l.ncs * l.code;
  l.off_misc = l.off_bar + (2 * ks::MAXST + 2 * ks::NBUF + 4 + 1) * 8;
  l.off_l = (l.off_misc + 32 + 15) / 16 * 16;
  l.total = l.off_l + 2 * ks::MAXN * 8 + 1024;
  return l;
}

// Position in a ring of n stages and the parity of its current phase.
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int n) {
    if (++st == n) {
      st = 0;
      ph ^= 1u;
    }
  }
};

// One CTA's walk over its share of the tiles.
struct Walk {
  int s, g, t, T, n;
};

template <int MODE>
__device__ __forceinline__ int ks_entries(const KeyScanParams& p, int s) {
  if (MODE == SCAN_WEIGHTS) return p.len ? min(max(__ldg(p.len + s), 0), p.L) : p.L;
  if (p.slice_seq) {
    const int t = __ldg(p.slice_seq + s);
    if (t < 0 || t >= p.n_seq) return 0;
  }
  const int n = max(__ldg(p.len + s), 0);
  return min(n / kPage + (n % kPage != 0), p.L);
}
// Tiles of one (slice, KV head); a slice without blocks still has its scores written.
template <int MODE>
__device__ __forceinline__ int ks_tiles(int n) {
  const int t = n / ks::BM + (n % ks::BM != 0);
  return MODE == SCAN_SCORES && t == 0 ? 1 : t;
}
template <int MODE>
__device__ __forceinline__ void ks_enter(const KeyScanParams& p, Walk& w) {
  w.n = ks_entries<MODE>(p, w.s);
  w.T = ks_tiles<MODE>(w.n);
}
template <int MODE>
__device__ __forceinline__ void ks_next(const KeyScanParams& p, Walk& w) {
  if (++w.t < w.T) return;
  w.t = 0;
  if (++w.g < p.Hkv) return;
  w.g = 0;
  do {
    ++w.s;
    if (w.s >= p.S) return;   // past the last triple: the caller has none left
    ks_enter<MODE>(p, w);
  } while (w.T == 0);
}

__device__ __forceinline__ float max_nan2(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

__device__ __forceinline__ float max_nan3(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ __forceinline__ void ks_wait_drain(uint64_t* b, uint32_t parity) {
  const unsigned long long t0 = globaltimer();
  while (!mbar_try_wait(b, parity)) {
    if (globaltimer() - t0 > kWaitLimitNs) return;
  }
}

// The MMA warp's wait: polls, so that the time limit holds to the poll.  The
// warp stays converged, and one elected lane issues: descriptors of a
// converged warp are kept in uniform registers.
__device__ __forceinline__ bool ks_poll(uint64_t* b, uint32_t parity, volatile int* abort, unsigned long long limit_ns) {
  if (__all_sync(0xffffffffu, mbar_test_wait(b, parity))) return true;
  const unsigned long long t0 = globaltimer();
  while (!__all_sync(0xffffffffu, mbar_test_wait(b, parity))) {
    const bool late = globaltimer() - t0 > limit_ns;
    if (__any_sync(0xffffffffu, late || *abort)) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t x;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(x));
  return x != 0;
}

// 16 bytes of pool codes -> 16-bit values of Q's type, as 16-byte words.
template <int KIND>
__device__ __forceinline__ void widen_chunk(const uint4& w, bool bf16, uint4 (&o)[KvChunk<KIND>::N / 8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  if constexpr (KIND == KV_I4) {
#pragma unroll
    for (int t = 0; t < 4; ++t) o[t] = widen_i4x8(u[t], bf16);
  } else {
    uint2 x[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if constexpr (KIND == KV_F8) {
        x[t] = widen_e4m3x4(u[t]);
        if (bf16) {   // every E4M3 value is a bf16 value
          const float2 a = f16x2_to_f2(x[t].x), b = f16x2_to_f2(x[t].y);
          x[t] = make_uint2(pack2h(a.x, a.y, true), pack2h(b.x, b.y, true));
        }
      } else {
        x[t] = widen_i8x4(u[t], bf16);
      }
    }
    o[0] = make_uint4(x[0].x, x[0].y, x[1].x, x[1].y);
    o[1] = make_uint4(x[2].x, x[2].y, x[3].x, x[3].y);
  }
}

// max(q, 0) or min(q, 0) of eight 16-bit values; a NaN stays one.
__device__ __forceinline__ uint4 sign_part(const uint4& x, bool plus, bool bf16) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
  uint32_t o[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (bf16) {
      const __nv_bfloat162 z = __floats2bfloat162_rn(0.f, 0.f), h = *reinterpret_cast<const __nv_bfloat162*>(&u[t]);
      const __nv_bfloat162 y = plus ? __hmax2_nan(h, z) : __hmin2_nan(h, z);
      o[t] = *reinterpret_cast<const uint32_t*>(&y);
    } else {
      const __half2 z = __floats2half2_rn(0.f, 0.f), h = *reinterpret_cast<const __half2*>(&u[t]);
      const __half2 y = plus ? __hmax2_nan(h, z) : __hmin2_nan(h, z);
      o[t] = *reinterpret_cast<const uint32_t*>(&y);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ float widen16(uint16_t x, bool bf16) {
  return bf16 ? __uint_as_float((uint32_t)x << 16) : __half2float(__ushort_as_half(x));
}

// One score from its definition, by a warp.  The two products of the tensor core
// put a zero against the bound that a component's sign does not use, and zero
// times infinity is NaN: so a block with an infinite bound (a key of a quantised
// pool beyond f16's range has one) comes out NaN where the score is a number.
// A warp that sees a NaN forms that score again: here a component takes the
// bound of its sign alone, and a zero takes none.  NaN where q or a bound is, or
// where infinite terms of both signs meet.  q: the slice's first vector of the
// KV head; hi, lo: the page's bounds.  Not inlined: hardly ever called.
template <int D>
__device__ __noinline__ float score_by_definition(const uint16_t* q, const uint16_t* hi, const uint16_t* lo, int NV, int G,
                                                  int Hq, bool bf16) {
  constexpr int PER = D / 32;
  const int d0 = (threadIdx.x & 31) * PER;
  const float NaN = __int_as_float(0x7fc00000);
  float h[PER], l[PER];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    h[i] = widen16(__ldg(hi + d0 + i), bf16);
    l[i] = widen16(__ldg(lo + d0 + i), bf16);
    bad = bad || h[i] != h[i] || l[i] != l[i];
  }
  if (__any_sync(0xffffffffu, bad)) return NaN;
  float best = __int_as_float(0xff800000);
  constexpr int B = 4;   // vectors a step, for their latencies to overlap
  for (int v0 = 0; v0 < NV; v0 += B) {
    double sum[B];       // finite bf16 products reach beyond fp32
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int v = min(v0 + b, NV - 1);
      const uint16_t* qv = q + (size_t)(v / G * Hq + v % G) * D + d0;
      sum[b] = 0.;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const float x = widen16(__ldg(qv + i), bf16);
        sum[b] += x > 0.f ? (double)x * h[i] : x < 0.f ? (double)x * l[i] : (double)x;
      }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
#pragma unroll
      for (int b = 0; b < B; ++b) sum[b] += __shfl_xor_sync(0xffffffffu, sum[b], o);
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      bad = bad || sum[b] != sum[b];
      best = fmaxf(best, (float)sum[b]);
    }
    if (bad) return NaN;
  }
  return best;
}
// The scores of a warp's keys (lane = key, page its pool page, there: it has one), NaNs looked at again.
template <int D>
__device__ __forceinline__ float settle_scores(const KeyScanParams& p, int s, int g, float score, int page, bool there) {
  for (unsigned nan = __ballot_sync(0xffffffffu, there && score != score); nan; nan &= nan - 1) {
    const int src = __ffs(nan) - 1;
    const size_t at = ((size_t)__shfl_sync(0xffffffffu, page, src) * p.Hkv + g) * D;
    const float x = score_by_definition<D>(static_cast<const uint16_t*>(p.q) + ((size_t)s * p.Nq * p.Hq + g * p.G) * D,
                                           static_cast<const uint16_t*>(p.k[0]) + at, static_cast<const uint16_t*>(p.k[1]) + at,
                                           p.NV, p.G, p.Hq, p.q_bf16 != 0);
    if ((int)(threadIdx.x & 31) == src) score = x;
  }
  return score;
}

template <int D, int MODE, int KIND>
__global__ void __launch_bounds__(ks::kThreads<KIND == KV_I8 || KIND == KV_I4 || KIND == KV_F8>, 1)
    keyscan_stream_kernel(const KeyScanParams p, int tma_ok, const __grid_constant__ CUtensorMap t0,
                          const __grid_constant__ CUtensorMap t1) {
  using namespace ks;
  constexpr bool QUANT = KIND == KV_I8 || KIND == KV_I4 || KIND == KV_F8;
  constexpr int NK = MODE == SCAN_SCORES ? 2 : 1;   // stages per tile
  constexpr int NKEY = kKeyWarps<QUANT>;
  constexpr int PARTS = kParts<D, NK>;
  constexpr int ATOM = BM * 128;                    // one 64-column atom of a key tile
  constexpr int KT = D / 64;
  const float INF = __int_as_float(0x7f800000);
  extern __shared__ unsigned char smem_raw[];
  // aligned by an offset, so that the compiler still knows the pointer for a shared one (plain, not generic, loads)
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const KsLayout ly = ks_layout<D, MODE, KIND>(p.NV);
  const int N = ly.N, NST = ly.nst;   // two groups of key warps: NST > NK (see kGroups)
  uint64_t* k_full = reinterpret_cast<uint64_t*>(sm + ly.off_bar);
  uint64_t* k_empty = k_full + MAXST;
  uint64_t* s_full = k_empty + MAXST;
  uint64_t* s_empty = s_full + NBUF;
  uint64_t* q_full = s_empty + NBUF;
  uint64_t* q_empty = q_full + 2;
  uint64_t* drain = q_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + ly.off_misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + ly.off_misc + 4);
  float* l2 = reinterpret_cast<float*>(sm + ly.off_l);            // [2][MAXN] lse in log2 units
  int* lim = reinterpret_cast<int*>(sm + ly.off_l) + 2 * MAXN;    // [2][MAXN] n_s-relative causal limits

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool bf16 = p.q_bf16 != 0;
  const unsigned long long wait_ns = p.wait_ns;

  // ---- this CTA's share of the triples: every warp adds up the slices' tile
  // counts, 8 slices a lane and step, and finds the slice of its first tile
  Walk w0;
  int mine;   // tiles of the share
  {
    constexpr int PER = 8;
    auto counts = [&](int base, int (&n)[PER], int (&c)[PER]) -> int {   // of 8 slices from base on; their sum
      int sum = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) n[i] = base + i < p.S ? ks_entries<MODE>(p, base + i) : 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        c[i] = base + i < p.S ? ks_tiles<MODE>(n[i]) * p.Hkv : 0;
        sum += c[i];
      }
      return sum;
    };
    int n[PER], c[PER], total = 0;
    if (MODE == SCAN_WEIGHTS && !p.len) {
      total = ks_tiles<MODE>(p.L) * p.Hkv * p.S;
    } else {
      for (int base = 0; base < p.S; base += 32 * PER) total += __reduce_add_sync(0xffffffffu, counts(base + lane * PER, n, c));
    }
    // even shares, the first total % CTAs of them one tile longer
    const int each = total / (int)gridDim.x, more = total % (int)gridDim.x, bid = (int)blockIdx.x;
    const int start = bid * each + min(bid, more);
    mine = each + (bid < more ? 1 : 0);
    if (mine == 0) return;
    int slice = 0, left = 0, len = p.L;   // the slice, and the share's start within it
    if (MODE == SCAN_WEIGHTS && !p.len) {
      const int per = ks_tiles<MODE>(p.L) * p.Hkv;
      slice = start / per;
      left = start % per;
    } else {
      int carry = 0;
      for (int base = 0; base < p.S; base += 32 * PER) {
        int x = counts(base + lane * PER, n, c);
        const int sum = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const int before = carry + x - sum;
        const unsigned who = __ballot_sync(0xffffffffu, start >= before && start < before + sum);
        if (who) {
          int at = before, found = 0;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            if (!found && start < at + c[i]) {
              found = 1;
              slice = base + lane * PER + i;
              left = start - at;
              len = n[i];
            }
            at += c[i];
          }
          const int src = __ffs(who) - 1;
          slice = __shfl_sync(0xffffffffu, slice, src);
          left = __shfl_sync(0xffffffffu, left, src);
          len = __shfl_sync(0xffffffffu, len, src);
          break;
        }
        carry += __shfl_sync(0xffffffffu, x, 31);
      }
    }
    w0.s = slice;
    w0.n = len;
    w0.T = ks_tiles<MODE>(len);
    w0.g = left / w0.T;
    w0.t = left % w0.T;
  }

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(k_full + i, NKEY / kGroups<D, NK, QUANT> * (QUANT ? 1 : 32));
      mbar_init(k_empty + i, 1);
    }
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(s_empty + i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, 1 + NEPI);   // the MMAs of its last tile, and the reduction warps
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  uint32_t ncols = 32;
  while ((int)ncols < NBUF * PARTS * N) ncols <<= 1;
  if (warp == W_MMA) {
    tmem_alloc(tmem_holder, ncols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;
  // Key warps of 16-bit pools: stages filled so far, and (the lane that issues
  // them) the stages whose last fill was TMA loads, with its phase parity.
  int fills = 0;
  unsigned tma_pend = 0, tma_par = 0;

  if (warp < NEPI) {
    // ------------------------------------------------------------ reduction
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // tensor-memory lane base of this warp: 32 * (warp % 4), in bits 16 up
    const int grp = warp >> 2, kid = tid & 127;          // this warpgroup's tiles: grp, grp + 2, ...
    // What a thread needs of its key beside the products: loaded one tile
    // ahead into one of two register sets, which the loop names in turn (a
    // copy from one to the other would wait for the load).
    struct Key {
      int row;
      unsigned short scale;
      float old;
    };
    auto load_key = [&](const Walk& x, Key& a) {
      const int j = x.t * BM + kid;
      a.row = -1;
      a.old = 0.f;
      if (j < x.n) {
        const int list = MODE == SCAN_SCORES && p.slice_seq ? __ldg(p.slice_seq + x.s) : x.s;
        a.row = __ldg(p.rows + (size_t)list * p.L + j);
        if (MODE == SCAN_WEIGHTS && p.decay != 0.f) a.old = __ldcg(p.out + ((size_t)x.s * p.Hkv + x.g) * p.L + j);
      }
    };
    auto live = [&](const Key& a) { return a.row >= 0 && (long long)a.row < p.R; };
    auto load_scale = [&](const Walk& x, Key& a) {
      if (QUANT) a.scale = live(a) ? __ldg(p.k_scale + ((size_t)(a.row >> 6) * p.Hkv + x.g) * kPage + (a.row & 63)) : (unsigned short)0;
    };
    Walk w = w0;
    int unit = 0, unit_seen = -1;
    // The queries of the current (slice, KV head) are in their buffer.
    auto have_queries = [&]() {
      if (unit == unit_seen) return true;
      unit_seen = unit;
      return (bool)__all_sync(0xffffffffu, mbar_wait(q_full + (unit & 1), (unit >> 1) & 1, abort_flag, wait_ns));
    };
    // Over one tile of the share, whichever warpgroup's; the next (slice, KV
    // head) begins after its last.  Both warpgroups count the query buffers so, and
    // each gives a buffer back when it has passed the last tile that uses it:
    // after seeing it full, since an arrival any earlier could fall into the
    // phase of the buffer's use before.
    auto pass = [&](int k, Walk& x) -> bool {
      const bool last = k + 1 == mine || x.t + 1 == x.T;
      if (last) {
        if (!have_queries()) return false;
        __syncwarp();
        if (lane == 0) mbar_arrive(q_empty + (unit & 1));
        ++unit;
      }
      if (k + 1 < mine) ks_next<MODE>(p, x);
      return true;
    };
    // one tile: its key in cur; the group's next tile's goes to nxt
    auto tile = [&](int k, Key& cur, Key& nxt) -> bool {
      const int b = k % NBUF, qb = unit & 1;
      const int j = w.t * BM + kid;
      float* out = p.out + ((size_t)w.s * p.Hkv + w.g) * p.L;
      Walk nx = w;
      if (k + 2 < mine) {
        ks_next<MODE>(p, nx);
        ks_next<MODE>(p, nx);
        load_key(nx, nxt);
      }
      if (!have_queries()) return false;
      if (!__all_sync(0xffffffffu, mbar_wait(s_full + b, (k / NBUF) & 1, abort_flag, wait_ns))) return false;
      tc_fence_after();
      const float4* l4 = reinterpret_cast<const float4*>(l2 + qb * MAXN);
      const int4* m4 = reinterpret_cast<const int4*>(lim + qb * MAXN);
      // causal: every query sees positions up to n - Nq
      const bool masked = MODE == SCAN_WEIGHTS && p.causal && w.t * BM + BM - 1 > w.n - p.Nq;
      const float cs = QUANT ? p.c * __half2float(__ushort_as_half(cur.scale)) : p.c;
      float r[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) r[u] = MODE == SCAN_SCORES ? -INF : 0.f;
      for (int c0 = 0; c0 < N; c0 += 16) {
        uint32_t x[16];
        tmem_ld16(tbase + lanes + b * PARTS * N + c0, x);
        if constexpr (PARTS == 2) {
          uint32_t y[16];
          tmem_ld16(tbase + lanes + (b * PARTS + 1) * N + c0, y);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) + __uint_as_float(y[i]));
        }
        if (MODE == SCAN_SCORES) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float m = max_nan2(r[i & 3], __uint_as_float(x[i]));
            r[i & 3] = c0 + i < p.NV ? m : r[i & 3];
          }
        } else {
          // Columns without a query, and queries that saw nothing, have
          // l = +inf and add nothing whatever their product.  Selections, not
          // branches: a branch per column made this loop the kernel's bound
          // (45.7 us where selections take 31, 4 x 16,384 entries).
          float e[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 l = l4[c0 / 4 + i];
            const float lv[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const float ex = fast_ex2(fmaf(__uint_as_float(x[4 * i + u]), cs, -lv[u]));
              e[4 * i + u] = lv[u] == INF ? 0.f : ex;
            }
          }
          if (masked) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int4 m = m4[c0 / 4 + i];
              e[4 * i] = j <= m.x ? e[4 * i] : 0.f;
              e[4 * i + 1] = j <= m.y ? e[4 * i + 1] : 0.f;
              e[4 * i + 2] = j <= m.z ? e[4 * i + 2] : 0.f;
              e[4 * i + 3] = j <= m.w ? e[4 * i + 3] : 0.f;
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) r[i & 3] += e[i];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_empty + b);
      if constexpr (MODE == SCAN_SCORES) {
        const float best = settle_scores<D>(p, w.s, w.g, max_nan2(max_nan2(r[0], r[1]), max_nan2(r[2], r[3])), cur.row,
                                            j < w.n && live(cur));
        if (j < w.n) out[j] = live(cur) ? best : -INF;
        // past the sequence's blocks: the (slice, KV head)'s last tile fills the rest
        if (w.t + 1 == w.T)
          for (int f = w.n + kid; f < p.L; f += 128) out[f] = -INF;
      } else if (j < w.n) {
        const float add = live(cur) ? (r[0] + r[1]) + (r[2] + r[3]) : 0.f;
        out[j] = p.decay == 0.f ? add : fmaf(p.decay, cur.old, add);
      }
      if (k + 2 < mine) load_scale(nx, nxt);
      return pass(k, w) && (k + 1 >= mine || pass(k + 1, w));
    };
    Key ka, kb;
    const bool begun = grp == 0 || pass(0, w);
    if (begun && grp < mine) {
      load_key(w, ka);
      load_scale(w, ka);
    }
    for (int k = grp; begun && k < mine; k += 4) {
      if (!tile(k, ka, kb)) break;
      if (k + 2 < mine && !tile(k + 2, kb, ka)) break;
    }
  } else if (warp == W_MMA) {
    // ------------------------------------------------------------ MMA issue
    const uint32_t id = make_idesc_f16(BM, N, bf16, false);
    const uint64_t dK = sdesc_sw128(smem_u32(sm + ly.off_k), 16, 1024);
    const uint64_t dQ = sdesc_sw128(smem_u32(sm + ly.off_q), 16, 1024);
    const uint32_t qatom = (uint32_t)N * 128;
    Walk w = w0;
    int unit = 0;
    bool ok = true;
    Ring kr, sr;
    for (int k = 0; ok && k < mine; ++k) {
      const int qb = unit & 1;
      const bool first = k == 0 || w.t == 0, last = k + 1 == mine || w.t + 1 == w.T;
      if (first) ok = ks_poll(q_full + qb, (unit >> 1) & 1, abort_flag, wait_ns);
      ok = ok && ks_poll(s_empty + sr.st, sr.ph ^ 1u, abort_flag, wait_ns);
#pragma unroll
      for (int m = 0; m < NK; ++m) {
        const int st = kr.st;
        ok = ok && ks_poll(k_full + st, kr.ph, abort_flag, wait_ns);
        if (!ok) break;
        kr.next(NST);
        tc_fence_after();
        const uint64_t a = sdesc_at(dK, st * ly.tile), q = sdesc_at(dQ, qb * ly.qb_bytes + m * KT * qatom);
        if (elect_one()) {
          fence_proxy_async_smem();   // the stage's cp.async copies arrived by themselves
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            mma_ss(tbase + (sr.st * PARTS + m % PARTS) * N, sdesc_at(a, (i >> 2) * ATOM + (i & 3) * 32),
                   sdesc_at(q, (i >> 2) * qatom + (i & 3) * 32), id, m >= PARTS || i > 0);
          tc_commit(k_empty + st);
          if (m == NK - 1) {
            tc_commit(s_full + sr.st);
            if (last) tc_commit(q_empty + qb);
          }
        }
        __syncwarp();
      }
      if (!ok) break;
      sr.next(NBUF);
      if (last) ++unit;
      if (k + 1 < mine) ks_next<MODE>(p, w);
    }
    if (elect_one()) {
      tc_commit(drain);
      ks_wait_drain(drain, 0);
    }
    __syncwarp();
  } else if (warp == W_Q) {
    // ------------------------------------------------------------ queries
    Walk w = w0;
    int left = mine;
    constexpr int CPR = D / 8;   // 16-byte chunks of a query vector
    for (int unit = 0; left > 0; ++unit) {
      const int qb = unit & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(q_empty + qb, ((unit >> 1) & 1) ^ 1, abort_flag, wait_ns))) break;
      unsigned char* dst = sm + ly.off_q + qb * ly.qb_bytes;
      const uint16_t* qg = static_cast<const uint16_t*>(p.q);
      const uint16_t* base = qg + ((size_t)w.s * p.Nq * p.Hq + w.g * p.G) * D;
      auto row_at = [&](int v) { return base + (size_t)(v / p.G * p.Hq + v % p.G) * D; };
      if (MODE == SCAN_WEIGHTS) {
        // all copies under way before the first is waited for: the first
        // tile's products wait for them
        for (int f = lane; f < N * CPR; f += 32) {
          const int v = f / CPR, c = f % CPR;
          cp_async16(dst + (c >> 3) * N * 128 + v * 128 + (((c & 7) ^ (v & 7)) << 4), row_at(min(v, p.NV - 1)) + c * 8, v < p.NV);
        }
      } else {
        for (int f0 = 0; f0 < N * CPR; f0 += 8 * 32) {   // N * CPR is a multiple of 128
          uint4 x[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int f = min(f0 + u * 32 + lane, N * CPR - 1), v = f / CPR;
            x[u] = __ldg(reinterpret_cast<const uint4*>(row_at(min(v, p.NV - 1))) + f % CPR);
          }
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int f = f0 + u * 32 + lane, v = f / CPR, c = f % CPR;
            if (f >= N * CPR) break;
            if (v >= p.NV) x[u] = make_uint4(0u, 0u, 0u, 0u);
            unsigned char* at = dst + (c >> 3) * N * 128 + v * 128 + (((c & 7) ^ (v & 7)) << 4);
            *reinterpret_cast<uint4*>(at) = sign_part(x[u], true, bf16);
            *reinterpret_cast<uint4*>(at + KT * N * 128) = sign_part(x[u], false, bf16);
          }
        }
      }
      if (MODE == SCAN_WEIGHTS) {
        for (int v = lane; v < N; v += 32) {
          const float l = v < p.NV ? __ldg(p.lse + ((size_t)w.s * p.Nq + v / p.G) * p.Hq + w.g * p.G + v % p.G) : -INF;
          l2[qb * MAXN + v] = l == -INF ? INF : l * kLog2e;
          lim[qb * MAXN + v] = w.n - p.Nq + v / p.G;
        }
        cp_async_wait_all();
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full + qb);
      // on to the next (slice, KV head) of the share
      const int here = w.T - w.t;
      left -= here;
      if (left > 0) {
        w.t = w.T - 1;
        ks_next<MODE>(p, w);
      }
    }
  } else {
    // ------------------------------------------------------------ keys
    constexpr int GROUPS = kGroups<D, NK, QUANT>, GW = NKEY / GROUPS, RW = BM / GW;   // warps of a group, rows of a warp
    const int grp = (warp - W_KEY) / GW, kw = (warp - W_KEY) % GW;
    // this group's tiles: grp, grp + GROUPS, ...; n_own of them
    const int n_own = (mine - grp + GROUPS - 1) / GROUPS;
    auto step = [&](Walk& x) {   // to the group's next tile (there is one)
#pragma unroll
      for (int i = 0; i < GROUPS; ++i) ks_next<MODE>(p, x);
    };
    Walk w = w0;
    Ring kr;
    if (grp == 1 && n_own > 0) {
      ks_next<MODE>(p, w);
#pragma unroll
      for (int i = 0; i < NK; ++i) kr.next(NST);
    }
    auto advance = [&]() {       // over the other group's stages
#pragma unroll
      for (int i = 0; i < (GROUPS - 1) * NK; ++i) kr.next(NST);
    };
    auto list_of_slice = [&](const Walk& x) {
      return MODE == SCAN_SCORES && p.slice_seq ? (size_t)max(__ldg(p.slice_seq + x.s), 0) : (size_t)x.s;
    };
    auto entry = [&](const Walk& x, int e) {   // list entry (page) of key e of the tile as it stands, -1 past the end
      const int j = x.t * BM + e;
      return j < x.n ? __ldg(p.rows + list_of_slice(x) * p.L + j) : -1;
    };
    auto row_of = [&](int r) { return r >= 0 && (long long)r < p.R ? r : -1; };
    if constexpr (!QUANT) {
      constexpr int CPR = D / 8;
      const int half = kw / (GW / 2), sub = kw % (GW / 2);   // 64-row half of the tile, RW rows of it
      // List entries PRE tiles ahead (a tile's share of HBM time is shorter
      // than the latency of a list load), in register sets that the unrolled
      // loop names in turn.
      int nx0[PRE], nx1[PRE];
      Walk wp = w;
      int kp = 0;
      auto fetch = [&](int& a, int& b) {
        if (kp < n_own) {
          a = entry(wp, half * 64 + lane);
          b = entry(wp, half * 64 + 32 + lane);
          if (++kp < n_own) step(wp);
        }
      };
#pragma unroll
      for (int i = 0; i < PRE; ++i) fetch(nx0[i], nx1[i]);
      bool ok = true;
      for (int k0 = 0; ok && k0 < n_own; k0 += PRE) {
#pragma unroll
        for (int i = 0; i < PRE; ++i) {
          if (!ok || k0 + i >= n_own) break;
          const int r0 = row_of(nx0[i]), r1 = row_of(nx1[i]), g = w.g;
          const int base = __shfl_sync(0xffffffffu, r0, 0);
          const bool run = __all_sync(0xffffffffu, r0 >= 0 && r0 == base + lane && r1 == base + 32 + lane) && tma_ok;
          const int own = sub * RW < 32 ? r0 : r1;   // the register that holds this warp's rows
#pragma unroll
          for (int m = 0; m < NK; ++m) {
            const int st = kr.st;
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(k_empty + st, kr.ph ^ 1u, abort_flag, wait_ns)))) break;
            unsigned char* dst = sm + ly.off_k + st * ly.tile + half * 64 * 128;
            tma_pend &= ~(1u << st);
            ++fills;
            if (run) {
              if (sub == 0 && lane == 0) {
                mbar_arrive_expect_tx(k_full + st, 64 * D * 2);
#pragma unroll
                for (int a = 0; a < KT; ++a) tma_load_3d(dst + a * ATOM, m ? &t1 : &t0, a * 64, g, base, k_full + st);
                tma_pend |= 1u << st;
                tma_par = (tma_par & ~(1u << st)) | (kr.ph << st);
              } else {
                mbar_arrive(k_full + st);
              }
            } else {
              const char* src = static_cast<const char*>(p.k[m]) + (size_t)g * (D * 2);
              const size_t pitch = (size_t)p.Hkv * (D * 2);
              unsigned char* mine_dst = dst + sub * RW * 128;
#pragma unroll
              for (int it = 0; it < RW * CPR / 32; ++it) {
                const int f = it * 32 + lane;
                const int e = f / CPR, c = f % CPR;   // row of the warp's RW, chunk
                const int r = __shfl_sync(0xffffffffu, own, (sub * RW + e) & 31);
                cp_async16(mine_dst + (c >> 3) * ATOM + e * 128 + (((c & 7) ^ (e & 7)) << 4), src + (r >= 0 ? r : 0) * pitch + c * 16,
                           r >= 0);
              }
              cp_async_mbar_arrive_noinc(k_full + st);
            }
            kr.next(NST);
          }
          advance();
          fetch(nx0[i], nx1[i]);
          if (k0 + i + 1 < n_own) step(w);
        }
      }
      cp_async_wait_all();
    } else {
      // RW rows of each of the group's tiles per warp; each lane copies, and
      // later widens, its own 16-byte chunks, which lie lane by lane in the code ring
      constexpr int CB = kv_row_bytes<KIND>(D), CPR = CB / 16, NIT = RW * CPR / 32;
      static_assert(RW * CPR % 32 == 0, "a warp's chunks fill its lanes");
      constexpr int AHEAD = ks_ahead<D, KIND>(), NCS = AHEAD + 1;
      unsigned char* ring = sm + ly.off_c + grp * NCS * ly.code + kw * RW * CB;
      Walk wi = w, wp = w;                          // the copies' walk, NCS tiles ahead; the list entries', PRE more
      int nx[PRE];                                  // rows of the next tiles to copy, lanes 0 .. RW - 1
      int ki = 0, kp = 0, slot = 0;
      auto fetch = [&](int& a) {
        if (kp < n_own) {
          a = entry(wp, kw * RW + lane % RW);
          if (++kp < n_own) step(wp);
        }
      };
#pragma unroll
      for (int i = 0; i < PRE; ++i) fetch(nx[i]);
      // the copies of tile ki, whose list entries are in `set`; one group, empty past the share
      auto issue = [&](int& set) {
        if (ki < n_own) {
          const int row = row_of(set), g = wi.g;
          unsigned char* dst = ring + slot * ly.code;
          if (++slot == NCS) slot = 0;
          const char* src = static_cast<const char*>(p.k[0]) + (size_t)g * CB + lane % CPR * 16;   // 32 % CPR = 0
          const size_t pitch = (size_t)p.Hkv * CB;
#pragma unroll
          for (int it = 0; it < NIT; ++it) {
            const int r = __shfl_sync(0xffffffffu, row, it * (32 / CPR) + lane / CPR);
            cp_async16(dst + (it * 32 + lane) * 16, src + (r >= 0 ? r : 0) * pitch, r >= 0);
          }
          fetch(set);
          if (++ki < n_own) step(wi);
        }
        cp_async_commit();
      };
      // one tile: widen it, issue the copies of the tile AHEAD later
      int rd = 0;
      auto tile = [&](int& set) -> bool {
        // copies of this tile have landed once at most AHEAD - 1 later groups are pending
        cp_async_wait<AHEAD - 1>();
        uint4 cw[NIT];
        const unsigned char* src = ring + rd * ly.code;
        if (++rd == NCS) rd = 0;
#pragma unroll
        for (int it = 0; it < NIT; ++it) cw[it] = *reinterpret_cast<const uint4*>(src + (it * 32 + lane) * 16);
        issue(set);   // into the slot that the tile before this one left
        const int st = kr.st;
        if (!__all_sync(0xffffffffu, mbar_wait(k_empty + st, kr.ph ^ 1u, abort_flag, wait_ns))) return false;
        kr.next(NST);
        advance();
        unsigned char* dst = sm + ly.off_k + st * ly.tile;
        constexpr int W = KvChunk<KIND>::N / 8;     // 16-byte words a chunk widens to
#pragma unroll
        for (int it = 0; it < NIT; ++it) {
          const int f = it * 32 + lane, e = kw * RW + f / CPR, c = (f % CPR) * W;
          uint4 o[W];
          widen_chunk<KIND>(cw[it], bf16, o);
#pragma unroll
          for (int x = 0; x < W; ++x)
            *reinterpret_cast<uint4*>(dst + ((c + x) >> 3) * ATOM + e * 128 + ((((c + x) & 7) ^ (e & 7)) << 4)) = o[x];
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full + st);
        return true;
      };
      static_assert(AHEAD <= PRE, "the list entries of the copies issued first");
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) issue(nx[i]);
      bool ok = true;
      for (int k0 = 0; ok && k0 < n_own; k0 += PRE) {
#pragma unroll
        for (int i = 0; i < PRE; ++i) {
          if (!ok || k0 + i >= n_own) break;
          ok = tile(nx[(i + AHEAD) % PRE]);
        }
      }
      cp_async_wait_all();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tbase, ncols);
  }
  if (*abort_flag) {   // final: every role has ended
    if (tid == 0 && p.err) atomicOr(p.err, FA_WS_WAIT_EXPIRED);
    if constexpr (!QUANT) {
      // No TMA load may still be writing when the CTA exits.  A stage's barrier
      // tells of its loads only once every warp of the group has arrived, so the
      // warps that gave up first arrive for the fills that others made after it.
      int* most = reinterpret_cast<int*>(l2);   // fills of each group's furthest warp
      constexpr int GROUPS = kGroups<D, NK, QUANT>, GW = NKEY / GROUPS;
      const int grp = (warp - W_KEY) / GW;
      if (tid < GROUPS) most[tid] = 0;
      __syncthreads();
      if (warp >= W_KEY && lane == 0) atomicMax(most + grp, fills);
      __syncthreads();
      if (warp >= W_KEY) {
        for (int u = fills; u < most[grp]; ++u) mbar_arrive(k_full + ((u / NK * GROUPS + grp) * NK + u % NK) % NST);
        for (int i = 0; i < NST; ++i)
          if ((tma_pend >> i) & 1u) ks_wait_drain(k_full + i, (tma_par >> i) & 1u);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Many query vectors (prompts): a CTA keeps its keys in shared memory and the
// queries stream past them.
//
// A CTA owns up to NT tiles of 128 keys, so that each staged query tile is
// used NT times; one warpgroup reduces each key tile (thread = key, as above)
// while the tensor core is at the others.  Each key tile has its own of the four
// accumulators.  Two warps issue the products, of alternate key tiles (weights) or
// query tiles (scores): an issued product holds its warp until the tensor core
// takes it, and the 300-odd clocks of one warp's waits and commits lie under
// the other's products.  Measured for a 2,048-token chunk over 16,384
// entries of 8 heads, D 128: NT 4 with 128 columns and one accumulator per key
// tile 229 us (1.13 PFLOP/s; the tensor core and the exponentials are each busy
// 53 % of the time); 64 columns and two accumulators 253 us; NT 3 with a
// fourth accumulator going round 247 us; 96 columns with five going round 272 us (a
// product costs about the same whatever its columns); a polynomial for 3 of
// 8 exponentials 345 us (the special-function units give 32 a clock and SM here).
// Scores (two stages per query tile, for max(q, 0) and min(q, 0)) keep both
// bounds of one key tile; a CTA walks several slices, and stages the bounds
// again only where the slice is of another sequence.
//   warps 0 .. 4 NT - 1   gather (and widen) the keys, then the reduction
//   then                  MMA issue; queries: TMA boxes of whole queries
//                         (weights), or loads split by sign (scores)
namespace kp {
template <int D, int MODE>
struct Shape {
  static constexpr bool SC = MODE == SCAN_SCORES;
  static constexpr int NT = SC ? 1 : D == 256 ? 2 : 4;      // key tiles
  static constexpr int N = D == 256 ? 64 : 128;             // query vectors per tile
  static constexpr int NBUF = 4;                            // accumulators
  static constexpr int NK = SC ? 2 : 1;                     // stages per query tile
  static constexpr int NST = SC ? (D == 256 ? 2 : 4) : D == 64 ? 4 : 2;
  static constexpr int NL = 4;                              // query tiles whose lse are on chip
  static constexpr int ATOM = ks::BM * 128;
  static constexpr int KMAT = ks::BM * D * 2;         // one matrix of one key tile
  static constexpr int QST = N * D * 2;               // one query stage
  // Issuing warps.  Scores of D 256 have one: two would need a pair of stages each.
  static constexpr int NMMA = SC && NST < 2 * NK ? 1 : 2;
  static constexpr int NEPI = 4 * NT, W_MMA = NEPI, W_Q = NEPI + NMMA, NQW = SC ? 8 : 1;
  static constexpr int THREADS = (W_Q + NQW) * 32;
  static constexpr int NQG = SC ? NST / NK : 1;            // groups of query warps
  static constexpr int OFF_Q = NT * NK * KMAT;
  static constexpr int OFF_BAR = OFF_Q + NST * QST;
  static constexpr int NBAR = 2 + 2 * NST + 2 * NBUF + NMMA + 2 * NL;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int OFF_L = (OFF_MISC + 16 + 15) / 16 * 16;     // [NL][N] lse, [NL][N] limits, [NL] flags
  static constexpr int OFF_IDX = OFF_L + (SC ? 0 : NL * N * 8 + NL * 4);
  static constexpr int OFF_ROW = OFF_IDX + NT * ks::BM * 4;        // [N] scores: query rows of a slice's first tile
  static constexpr int USED = OFF_ROW + (SC ? N * 4 : 0);
  static constexpr int SMEM = USED + 1024;
  static constexpr int PARTS = ks::kParts<D, NK>;
  static constexpr uint32_t COLS = NBUF * PARTS * N;
  static_assert(COLS <= 512 && (COLS & (COLS - 1)) == 0 && NBUF >= NT && NBUF == 4, "tensor memory");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};
}  // namespace kp

struct PromptPlan {
  int PT, q_box;    // weights: queries per tile, and per TMA box
  int nb, tiles;    // batches of key tiles per (slice, KV head), and key tiles of a list of L entries
  int sc, chunks;   // slices per CTA, chunks of slices
};

template <int D, int MODE, int KIND>
__global__ void __launch_bounds__((kp::Shape<D, MODE>::THREADS), 1)
    keyscan_prompt_kernel(const KeyScanParams p, const PromptPlan pl, const __grid_constant__ CUtensorMap tq) {
  using Sh = kp::Shape<D, MODE>;
  constexpr bool QUANT = KIND == KV_I8 || KIND == KV_I4 || KIND == KV_F8;
  constexpr int NT = Sh::NT, N = Sh::N, NBUF = Sh::NBUF, NMMA = Sh::NMMA, NK = Sh::NK, NST = Sh::NST, NL = Sh::NL, KT = D / 64;
  constexpr int BM = ks::BM;
  const float INF = __int_as_float(0x7f800000);
  extern __shared__ unsigned char smem_raw[];
  // aligned by an offset, so that the compiler still knows the pointer for a shared one (plain, not generic, loads)
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* key_full = reinterpret_cast<uint64_t*>(sm + Sh::OFF_BAR);
  uint64_t* key_seen = key_full + 1;     // both issuing warps have seen key_full's last phase
  uint64_t* q_full = key_seen + 1;
  uint64_t* q_empty = q_full + NST;
  uint64_t* s_full = q_empty + NST;
  uint64_t* s_empty = s_full + NBUF;
  uint64_t* drain = s_empty + NBUF;
  uint64_t* l_full = drain + NMMA;       // [NL] lse, limits and flag of a query tile
  uint64_t* l_empty = l_full + NL;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + Sh::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + Sh::OFF_MISC + 4);
  float* nl2 = reinterpret_cast<float*>(sm + Sh::OFF_L);   // minus lse, in log2 units; -inf adds nothing
  int* lim = reinterpret_cast<int*>(nl2 + NL * N);
  int* odd = lim + NL * N;               // a column of the tile adds nothing, whatever its product
  int* idx = reinterpret_cast<int*>(sm + Sh::OFF_IDX);
  int* qrow = reinterpret_cast<int*>(sm + Sh::OFF_ROW);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool bf16 = p.q_bf16 != 0;
  const unsigned long long wait_ns = p.wait_ns;
  // (KV head, slice chunk) fastest: neighbouring CTAs read the same rows' heads
  const int per = p.Hkv * pl.chunks;
  const int batch = blockIdx.x / per, g = blockIdx.x % per % p.Hkv, chunk = blockIdx.x % per / p.Hkv;
  const int s_lo = chunk * pl.sc, s_hi = min(s_lo + pl.sc, p.S);
  const int nt = MODE == SCAN_SCORES ? (p.NV + N - 1) / N : (p.Nq + pl.PT - 1) / pl.PT;
  // This batch's key tiles, at most NT of them
  const int tile0 = (int)((long long)batch * pl.tiles / pl.nb);
  const int tile_end = (int)((long long)(batch + 1) * pl.tiles / pl.nb);
  const int j0 = tile0 * BM;                                       // its first key
  // The query tiles it takes of a slice of n entries: under a causal limit
  // from the first one that sees its first key on; none where n <= j0.
  auto first_tile = [&](int n) {
    if (j0 >= n) return nt;
    return MODE == SCAN_WEIGHTS && p.causal ? min(nt, max(0, j0 - (n - p.Nq)) / pl.PT) : 0;
  };
  // Accumulators of each key tile, as a power of two: all four for one, two each
  // for two, else one.  (By the batch's own number of tiles instead of the most
  // it can have: 236 us for 229 in the case above.)
  constexpr int bpt = NT == 1 ? 2 : NT == 2 ? 1 : 0;
  auto buffer = [&](int kt, int round) { return (kt << bpt) + (round & ((1 << bpt) - 1)); };
  auto key_tiles = [&](int n) { return min(tile_end - tile0, (n - j0 + BM - 1) / BM); };   // for n > j0
  if (MODE == SCAN_WEIGHTS && j0 >= ks_entries<MODE>(p, s_lo)) return;

  if (tid == 0) {
    mbar_init(key_full, Sh::NEPI * 32);
    mbar_init(key_seen, NMMA);
    for (int i = 0; i < NST; ++i) {
      mbar_init(q_full + i, Sh::NQW / Sh::NQG);
      mbar_init(q_empty + i, MODE == SCAN_SCORES ? 1 : NMMA);
    }
    for (int i = 0; i < NL; ++i) {
      mbar_init(l_full + i, 1);
      mbar_init(l_empty + i, Sh::NEPI);
    }
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(s_empty + i, 4);
    }
    for (int i = 0; i < NMMA; ++i) mbar_init(drain + i, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == Sh::W_MMA) {
    tmem_alloc(tmem_holder, Sh::COLS);
    tmem_relinquish();
  }
  if (MODE == SCAN_SCORES && tid < N) qrow[tid] = tid / p.G * p.Hq + tid % p.G;
  if (MODE == SCAN_WEIGHTS && pl.q_box * p.G < N) {
    // rows of a query tile that no box writes
    for (int f = tid; f < NST * Sh::QST / 16; f += Sh::THREADS)
      reinterpret_cast<uint4*>(sm + Sh::OFF_Q)[f] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;
  unsigned pend = 0, par = 0;   // weights, the lane that loads queries: stages with a TMA load, and its phase parity
  // the list (page table row) of a slice
  auto list_of_slice = [&](int s) { return MODE == SCAN_SCORES && p.slice_seq ? __ldg(p.slice_seq + s) : s; };

  if (warp < Sh::NEPI) {
    // ------------------------------------------------------------ keys and reduction
    const int kt = warp >> 2;                              // this warpgroup's key tile
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const int e = tid & 127;
    const int j = kt < tile_end - tile0 ? j0 + kt * BM + e : p.L;   // past every entry where the batch has no such tile
    // Each warp stages its own 32 keys, so that no barrier between warps stands
    // behind a wait that some of them may have given up.
    const int key0 = (warp & 3) * 32;
    int* my_idx = idx + kt * BM + key0;
    unsigned char* kdst = sm + kt * NK * Sh::KMAT + key0 * 128;   // 32 rows are four whole swizzle periods
    int loaded = -1, loads = 0, row = -1;
    float cs = p.c;
    int round = 0, lround = 0;                             // query tiles and lse slots so far
    bool ok = true;
    for (int s = s_lo; ok && s < s_hi; ++s) {
      const int n = ks_entries<MODE>(p, s);
      const int T = nt - first_tile(n);
      float* out = p.out + ((size_t)s * p.Hkv + g) * p.L;
      if (MODE == SCAN_SCORES && T == 0) {                 // no such blocks
        if (j < p.L) out[j] = -INF;
        continue;
      }
      const int list = list_of_slice(s);
      if (list != loaded) {
        // This warpgroup's key tile: its products of earlier slices have all
        // been read, so nothing else uses the tile; but an issuing warp that had
        // none of them may not have looked at key_full since.  For scores every
        // page of the table is staged, since later slices may see more of them.
        if (loads > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait(key_seen, (loads - 1) & 1, abort_flag, wait_ns)))) break;
        ++loads;
        loaded = list;
        row = j < (MODE == SCAN_SCORES ? p.L : n) ? __ldg(p.rows + (size_t)list * p.L + j) : -1;
        row = row >= 0 && (long long)row < p.R ? row : -1;
        my_idx[lane] = row;
        __syncwarp();
        if constexpr (QUANT) {
          constexpr int CB = kv_row_bytes<KIND>(D), CPR = CB / 16, W = KvChunk<KIND>::N / 8;
          constexpr int B = CPR < 8 ? CPR : 8;   // chunks per thread and step, all loaded before any is widened
          const char* src = static_cast<const char*>(p.k[0]) + (size_t)g * CB;
          const size_t pitch = (size_t)p.Hkv * CB;
          for (int f0 = lane; f0 < 32 * CPR; f0 += B * 32) {
            uint4 y[B];
#pragma unroll
            for (int u = 0; u < B; ++u) {
              const int f = f0 + u * 32, r = my_idx[f / CPR];
              y[u] = r >= 0 ? __ldg(reinterpret_cast<const uint4*>(src + r * pitch) + f % CPR) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u < B; ++u) {
              const int f = f0 + u * 32, k = f / CPR, c = f % CPR;
              uint4 o[W];
              widen_chunk<KIND>(y[u], bf16, o);
#pragma unroll
              for (int x = 0; x < W; ++x) {
                const int cc = c * W + x;
                *reinterpret_cast<uint4*>(kdst + (cc >> 3) * Sh::ATOM + k * 128 + (((cc & 7) ^ (k & 7)) << 4)) = o[x];
              }
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(key_full);
          if (row >= 0) cs = p.c * kv_scale_of(p.k_scale, row, g, p.Hkv);
        } else {
          constexpr int CPR = D / 8;
#pragma unroll
          for (int m = 0; m < NK; ++m) {
            const char* src = static_cast<const char*>(p.k[m]) + (size_t)g * (D * 2);
            const size_t pitch = (size_t)p.Hkv * (D * 2);
#pragma unroll 8
            for (int f = lane; f < 32 * CPR; f += 32) {
              const int k = f / CPR, c = f % CPR, r = my_idx[k];
              cp_async16(kdst + m * Sh::KMAT + (c >> 3) * Sh::ATOM + k * 128 + (((c & 7) ^ (k & 7)) << 4),
                         src + max(r, 0) * pitch + c * 16, r >= 0);
            }
          }
          cp_async_mbar_arrive_noinc(key_full);
        }
      }
      float old = 0.f;
      if (MODE == SCAN_WEIGHTS && p.decay != 0.f && j < n) old = __ldcg(out + j);
      float total = MODE == SCAN_SCORES ? -INF : 0.f, total2 = -INF;   // scores: their maximum is the result
      const int kn = T > 0 ? key_tiles(n) : 0;
      for (int t = 0; t < T; ++t) {
        const int sl = lround % NL;
        if (MODE == SCAN_WEIGHTS) {
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(l_full + sl, (lround / NL) & 1, abort_flag, wait_ns)))) break;
          ++lround;
        }
        const int b = buffer(kt, round), phase = (round >> bpt) & 1;
        ++round;
        if (kt >= kn) {   // no such key tile
          __syncwarp();
          if (MODE == SCAN_WEIGHTS && lane == 0) mbar_arrive(l_empty + sl);
          continue;
        }
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(s_full + b, phase, abort_flag, wait_ns)))) break;
        tc_fence_after();
        const uint32_t at = tbase + lanes + b * Sh::PARTS * N;
        const int m = p.NV - t * N;      // scores: real columns of the tile
        const float4* l4 = reinterpret_cast<const float4*>(nl2 + sl * N);
        const int4* m4 = reinterpret_cast<const int4*>(lim + sl * N);
        // this warp's highest key against the tile's first query
        const bool masked = MODE == SCAN_WEIGHTS && (odd[sl] || (p.causal && j0 + kt * BM + (warp & 3) * 32 + 31 > lim[sl * N]));
        float2 r0 = make_float2(0.f, 0.f), r1 = r0;
        const float2 cs2 = make_float2(cs, cs);
        // 32 columns at a time, the next ones' load under way meanwhile
        uint32_t x[2][32];
        if constexpr (Sh::PARTS == 1) tmem_ld32(at, x[0]);
#pragma unroll
        for (int c = 0; c < N / 32; ++c) {
          uint32_t(&y)[32] = x[Sh::PARTS == 2 ? 0 : c & 1];
          if constexpr (Sh::PARTS == 2) {
            tmem_ld32_nowait(at + 32 * c, y);
            tmem_ld32_nowait(at + N + 32 * c, x[1]);
            tmem_wait_ld_tied(y);
            tmem_wait_ld_tied(x[1]);
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) + __uint_as_float(x[1][i]));
          } else if (c > 0) {
            tmem_wait_ld_tied(y);
          }
          if (c + 1 < N / 32) {
            if constexpr (Sh::PARTS == 1) tmem_ld32_nowait(at + 32 * (c + 1), x[(c + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_empty + b);
          }
          if constexpr (MODE == SCAN_SCORES) {
            if (m >= N) {
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                total = max_nan3(total, __uint_as_float(y[i]), __uint_as_float(y[i + 1]));
                total2 = max_nan3(total2, __uint_as_float(y[i + 2]), __uint_as_float(y[i + 3]));
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float z = max_nan2(total, __uint_as_float(y[i]));
                total = 32 * c + i < m ? z : total;
              }
            }
          } else if (!masked) {
            // two columns at a time
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 l = l4[8 * c + i];
              const float2 a = __ffma2_rn(make_float2(__uint_as_float(y[4 * i]), __uint_as_float(y[4 * i + 1])), cs2,
                                          make_float2(l.x, l.y));
              const float2 d = __ffma2_rn(make_float2(__uint_as_float(y[4 * i + 2]), __uint_as_float(y[4 * i + 3])), cs2,
                                          make_float2(l.z, l.w));
              r0 = __fadd2_rn(r0, make_float2(fast_ex2(a.x), fast_ex2(a.y)));
              r1 = __fadd2_rn(r1, make_float2(fast_ex2(d.x), fast_ex2(d.y)));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 l = l4[8 * c + i];
              const int4 q = m4[8 * c + i];
              const float lv[4] = {l.x, l.y, l.z, l.w};
              const int mv[4] = {q.x, q.y, q.z, q.w};
              float ev[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const float ex = fast_ex2(fmaf(__uint_as_float(y[4 * i + u]), cs, lv[u]));
                ev[u] = lv[u] == -INF || j > mv[u] ? 0.f : ex;
              }
              r0 = __fadd2_rn(r0, make_float2(ev[0], ev[1]));
              r1 = __fadd2_rn(r1, make_float2(ev[2], ev[3]));
            }
          }
        }
        if (MODE == SCAN_WEIGHTS) {
          __syncwarp();
          if (lane == 0) mbar_arrive(l_empty + sl);
          total += (r0.x + r0.y) + (r1.x + r1.y);
        }
      }
      if (!QUANT) cp_async_wait_all();   // also where no query tile sees these keys
      if constexpr (MODE == SCAN_SCORES) total = settle_scores<D>(p, s, g, max_nan2(total, total2), row, ok && j < n && row >= 0);
      if (j < n) {
        if (MODE == SCAN_SCORES) {
          out[j] = row >= 0 ? total : -INF;
        } else {
          const float add = row >= 0 ? total : 0.f;
          out[j] = p.decay == 0.f ? add : fmaf(p.decay, old, add);
        }
      } else if (MODE == SCAN_SCORES && j < p.L) {
        out[j] = -INF;
      }
    }
  } else if (warp < Sh::W_Q) {
    // ------------------------------------------------------------ MMA issue
    const int mw = warp - Sh::W_MMA;
    const uint32_t id = make_idesc_f16(BM, N, bf16, false);
    const uint64_t dK = sdesc_sw128(smem_u32(sm), 16, 1024);
    const uint64_t dQ = sdesc_sw128(smem_u32(sm + Sh::OFF_Q), 16, 1024);
    bool ok = true;
    int loaded = -1, loads = 0, round = 0;
    // The products of stage st (part m of a query tile) with key tile kt
    auto product = [&](int kt, int m, int st) -> bool {
      const int b = buffer(kt, round);
      if (m == 0 && !ks_poll(s_empty + b, ((round >> bpt) & 1) ^ 1, abort_flag, wait_ns)) return false;
      tc_fence_after();
      const uint64_t a = sdesc_at(dK, (kt * NK + m) * Sh::KMAT), q = sdesc_at(dQ, st * Sh::QST);
      if (elect_one()) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          mma_ss(tbase + (b * Sh::PARTS + m % Sh::PARTS) * N, sdesc_at(a, (i >> 2) * Sh::ATOM + (i & 3) * 32),
                 sdesc_at(q, (i >> 2) * (N * 128) + (i & 3) * 32), id, m >= Sh::PARTS || i > 0);
        if (m == NK - 1) tc_commit(s_full + b);
      }
      __syncwarp();
      return true;
    };
    for (int s = s_lo; ok && s < s_hi; ++s) {
      const int n = ks_entries<MODE>(p, s);
      const int T = nt - first_tile(n);
      if (T == 0 && MODE == SCAN_SCORES) continue;
      const int kn = T > 0 ? key_tiles(n) : 0;
      const int list = list_of_slice(s);
      if (list != loaded) {
        loaded = list;
        ok = ks_poll(key_full, loads & 1, abort_flag, wait_ns);
        ++loads;
        if (ok && lane == 0) mbar_arrive(key_seen);
        fence_proxy_async_smem();   // the keys' cp.async copies arrived by themselves
      }
      for (int t = 0; ok && t < T; ++t, ++round) {
        if (MODE == SCAN_SCORES && NMMA == 2 && (round & 1) != mw) continue;   // the other warp's query tile, and its stages
#pragma unroll
        for (int m = 0; m < NK; ++m) {
          const int use = round * NK + m, st = use % NST;
          if (!(ok = ks_poll(q_full + st, (use / NST) & 1, abort_flag, wait_ns))) break;
          if (MODE == SCAN_SCORES) {
            ok = product(0, m, st);
          } else {
#pragma unroll
            for (int kt = 0; kt < NT; kt += NMMA)
              if (ok && kt + mw < kn) ok = product(kt + mw, m, st);
          }
          if (!ok) break;
          if (elect_one()) tc_commit(q_empty + st);
          __syncwarp();
        }
      }
    }
    if (elect_one()) {
      tc_commit(drain + mw);
      ks_wait_drain(drain + mw, 0);
    }
    __syncwarp();
  } else if (MODE == SCAN_WEIGHTS) {
    // ------------------------------------------------------------ queries by TMA
    const int s = s_lo, n = ks_entries<MODE>(p, s), PT = pl.PT;
    const int t0 = first_tile(n), T = nt - t0;
    // This lane's columns v = lane + 32 u of a query tile: query v / G, head v % G.
    // The next tile's lse are loaded as they stand and looked at when it is that tile's turn.
    const float* lse_at[N / 32];
    int qi[N / 32];
    float raw[N / 32];
#pragma unroll
    for (int u = 0; u < N / 32; ++u) {
      const int v = lane + 32 * u;
      qi[u] = v < PT * p.G ? t0 * PT + v / p.G : 0x3fffffff;   // past every query
      lse_at[u] = p.lse + (size_t)s * p.Nq * p.Hq + g * p.G + v % p.G;
    }
    auto load_lse = [&]() {
#pragma unroll
      for (int u = 0; u < N / 32; ++u) raw[u] = __ldg(lse_at[u] + (size_t)min(qi[u], p.Nq - 1) * p.Hq);
    };
    load_lse();
    for (int t = 0; t < T; ++t) {
      const int st = t % NST, u2 = t / NST, sl = t % NL;
      if (!__all_sync(0xffffffffu, mbar_wait(q_empty + st, (u2 & 1) ^ 1, abort_flag, wait_ns))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full + st, (uint32_t)KT * pl.q_box * p.G * 128u);
#pragma unroll
        for (int a = 0; a < KT; ++a)
          tma_load_3d(sm + Sh::OFF_Q + st * Sh::QST + a * N * 128, &tq, a * 64, g * p.G, s * p.Nq + (t0 + t) * PT, q_full + st);
        pend |= 1u << st;
        par = (par & ~(1u << st)) | ((unsigned)(u2 & 1) << st);
      }
      __syncwarp();
      if (!__all_sync(0xffffffffu, mbar_wait(l_empty + sl, ((t / NL) & 1) ^ 1, abort_flag, wait_ns))) break;
      bool hide = false;
#pragma unroll
      for (int u = 0; u < N / 32; ++u) {
        const int v = lane + 32 * u;
        const float l = qi[u] >= p.Nq || raw[u] == -INF ? -INF : raw[u] * -kLog2e;
        nl2[sl * N + v] = l;
        lim[sl * N + v] = p.causal ? n - p.Nq + min(qi[u], p.Nq) : 0x7fffffff;
        hide = hide || !(l > -INF);
        if (qi[u] < 0x3fffffff) qi[u] += PT;
      }
      load_lse();
      hide = __any_sync(0xffffffffu, hide);
      if (lane == 0) odd[sl] = hide;
      __syncwarp();
      if (lane == 0) mbar_arrive(l_full + sl);
    }
  } else {
    // ------------------------------------------------------------ queries, split by sign
    // Two groups of four warps on alternate query tiles, each with a pair of
    // stages of its own (and an issuing warp that it alone feeds): the waits and
    // fences of one lie under the other's stores (16 x 128 queries, 1,562 blocks:
    // 54 us, 58 with all eight warps at every tile; 55 since the keys are staged by
    // warps).  At D 256 one group of
    // eight, as there is one pair.  Measured besides: the bounds in tensor
    // memory instead of shared memory, 55 us (a query tile 0.70 us for 0.76, but
    // a CTA starts 1 us later); all eight warps with two tiles of loads in
    // flight, 61 us.
    constexpr int CPR = D / 8, GW = Sh::NQW / Sh::NQG, STEP = GW * 32, NX = N * CPR / STEP;
    const int grp = (warp - Sh::W_Q) / GW, qt = (tid - Sh::W_Q * 32) % STEP;
    const uint16_t* qg = static_cast<const uint16_t*>(p.q);
    // This thread's 16-byte words of a query tile.  qrow holds the query rows
    // (query * Hq + head) of a slice's first tile; where whole queries fill a
    // tile, the rows of tile t are t * pitch further on.
    uint4 x[NX];
    const int pitch = N / p.G * p.Hq;
    auto fetch = [&](int s, int t) {
      const uint16_t* base = qg + ((size_t)s * p.Nq * p.Hq + g * p.G) * D + (qt % CPR) * 8;   // STEP is a multiple of CPR
      if (N % p.G == 0 && (t + 1) * N <= p.NV) {
        base += (size_t)t * pitch * D;
#pragma unroll
        for (int i = 0; i < NX; ++i) x[i] = __ldg(reinterpret_cast<const uint4*>(base + (size_t)qrow[(i * STEP + qt) / CPR] * D));
      } else {   // past the last query: zeros
#pragma unroll
        for (int i = 0; i < NX; ++i) {
          const int v = t * N + (i * STEP + qt) / CPR;
          x[i] = v < p.NV ? __ldg(reinterpret_cast<const uint4*>(base + (size_t)(v / p.G * p.Hq + v % p.G) * D))
                           : make_uint4(0u, 0u, 0u, 0u);
        }
      }
    };
    // over the query tiles of all slices that have such blocks
    int s = s_lo, t = 0;
    auto enter = [&]() {
      while (s < s_hi && first_tile(ks_entries<MODE>(p, s)) == nt) ++s;
    };
    auto next = [&]() {
      if (++t < nt) return;
      t = 0;
      ++s;
      enter();
    };
    enter();
    for (int i = 0; i < grp; ++i) next();
    if (s < s_hi) fetch(s, t);
    bool ok = true;
    for (int k = 0; ok && s < s_hi; ++k) {
#pragma unroll
      for (int i = 0; i < Sh::NQG; ++i) next();
#pragma unroll
      for (int m = 0; m < NK; ++m) {
        const int st = grp * NK + m;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(q_empty + st, (k & 1) ^ 1, abort_flag, wait_ns)))) break;
        unsigned char* dst = sm + Sh::OFF_Q + st * Sh::QST;
#pragma unroll
        for (int i = 0; i < NX; ++i) {
          const int f = i * STEP + qt, r = f / CPR, c = f % CPR;
          *reinterpret_cast<uint4*>(dst + (c >> 3) * (N * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = sign_part(x[i], m == 0, bf16);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full + st);
      }
      if (s < s_hi) fetch(s, t);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == Sh::W_MMA) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tbase, Sh::COLS);
  }
  if (*abort_flag) {   // final: every role has ended
    if (tid == 0 && p.err) atomicOr(p.err, FA_WS_WAIT_EXPIRED);
    // No TMA load may still be writing when the CTA exits.  The lane that issued
    // a stage's loads makes its only arrival, so the loads alone are waited for.
    for (int i = 0; i < NST; ++i)
      if ((pend >> i) & 1u) ks_wait_drain(q_full + i, (par >> i) & 1u);
  }
}

// ---------------------------------------------------------------------------
// host side

bool ks_map(CUtensorMap* m, const void* base, bool bf16, int D, int Hkv, long long R) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hkv, (cuuint64_t)R};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * Hkv * 2};
  const cuuint32_t box[3] = {64, 1, 64};
  return tmap_encode_3d(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, dims, strides,
                        box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, int MODE, int KIND>
cudaError_t ks_stream(const KeyScanParams& p, cudaStream_t st) {
  auto kern = keyscan_stream_kernel<D, MODE, KIND>;
  const KsLayout ly = ks_layout<D, MODE, KIND>(p.NV);
  constexpr int NK = MODE == SCAN_SCORES ? 2 : 1;
  constexpr bool QUANT = KIND == KV_I8 || KIND == KV_I4 || KIND == KV_F8;
  if (ly.nst < 1 || (ks::kGroups<D, NK, QUANT> == 2 && ly.nst <= NK) || ly.total > 227 * 1024) return cudaErrorInvalidConfiguration;
  const cudaError_t e = once_per_device<3>(
      [kern] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ks::SMEM_MAX); });
  if (e != cudaSuccess) return e;
  CUtensorMap t0, t1;
  memset(&t0, 0, sizeof(t0));
  memset(&t1, 0, sizeof(t1));
  int tma = 0;
  if (!QUANT && p.R >= 64) {
    tma = 1;
    if (!ks_map(&t0, p.k[0], p.q_bf16 != 0, D, p.Hkv, p.R)) return cudaErrorInvalidValue;
    if (MODE == SCAN_SCORES && !ks_map(&t1, p.k[1], p.q_bf16 != 0, D, p.Hkv, p.R)) return cudaErrorInvalidValue;
  }
  const long long most = (long long)p.S * p.Hkv * ((p.L + ks::BM - 1) / ks::BM);
  const int sms = sm_count();
  const int grid = (int)(most < sms ? most : sms);
  kern<<<grid, ks::kThreads<QUANT>, ly.total, st>>>(p, tma, t0, t1);
  return cudaGetLastError();
}

template <int D, int MODE, int KIND>
cudaError_t ks_prompt(const KeyScanParams& p, cudaStream_t st) {
  using Sh = kp::Shape<D, MODE>;
  auto kern = keyscan_prompt_kernel<D, MODE, KIND>;
  const cudaError_t e = once_per_device<4>(
      [kern] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM); });
  if (e != cudaSuccess) return e;
  CUtensorMap tq;
  memset(&tq, 0, sizeof(tq));
  PromptPlan pl;
  memset(&pl, 0, sizeof(pl));
  pl.sc = 1;
  const int tiles = (p.L + ks::BM - 1) / ks::BM;
  pl.tiles = tiles;
  const long long slots = sm_count();
  if (MODE == SCAN_WEIGHTS) {
    pl.PT = Sh::N / p.G;
    const long long queries = (long long)p.S * p.Nq;
    pl.q_box = (int)(queries < pl.PT ? queries : pl.PT);
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hq, (cuuint64_t)queries};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * p.Hq * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)pl.q_box};
    if (!tmap_encode_3d(&tq, p.q_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p.q, dims,
                        strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
    // Batches of at most NT key tiles per (slice, KV head): as many as fill
    // the rounds of CTAs that full batches would take, so that the last round
    // is a full one of smaller batches.
    const long long units = (long long)p.S * p.Hkv;
    const int full = (tiles + Sh::NT - 1) / Sh::NT;
    const long long rounds = (units * full + slots - 1) / slots;
    const long long nb = rounds * slots / units;
    pl.nb = (int)(nb < full ? full : nb > tiles ? tiles : nb);
  } else {
    // Slices that share a sequence share its staged bounds.  The number of
    // slices a CTA walks is the one that gives the fewest query tiles per SM,
    // with the staging and start of a CTA counted as five of them.
    pl.nb = tiles;
    const long long units = (long long)p.Hkv * tiles, per_slice = (p.NV + Sh::N - 1) / Sh::N;
    long long best = -1;
    for (int sc = 1; sc <= p.S && sc <= 64; ++sc) {
      const long long ctas = units * ((p.S + sc - 1) / sc);
      const long long cost = (ctas + slots - 1) / slots * (sc * per_slice + 5);
      if (best < 0 || cost < best) {
        best = cost;
        pl.sc = sc;
      }
    }
  }
  pl.chunks = (p.S + pl.sc - 1) / pl.sc;
  const long long grid = (long long)pl.nb * p.Hkv * pl.chunks;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  kern<<<(unsigned)grid, Sh::THREADS, Sh::SMEM, st>>>(p, pl, tq);
  return cudaGetLastError();
}

template <int D, int MODE, int KIND>
cudaError_t ks_launch(const KeyScanParams& p, cudaStream_t st) {
  constexpr bool QUANT = KIND == KV_I8 || KIND == KV_I4 || KIND == KV_F8;
  constexpr int most = ks::kStreamVec<D, MODE == SCAN_SCORES ? 2 : 1, QUANT>;
  return p.NV <= most ? ks_stream<D, MODE, KIND>(p, st) : ks_prompt<D, MODE, KIND>(p, st);
}

template <int KIND>
cudaError_t ks_weights_kind(const KeyScanParams& p, int D, cudaStream_t st) {
  if (D == 64) return ks_launch<64, SCAN_WEIGHTS, KIND>(p, st);
  if (D == 128) return ks_launch<128, SCAN_WEIGHTS, KIND>(p, st);
  return ks_launch<256, SCAN_WEIGHTS, KIND>(p, st);
}

}  // namespace

// A query tile of the prompt form holds whole queries (64 vectors at D 256, else 128).
bool keyscan_supported(int D, int G) { return (D == 64 || D == 128 || D == 256) && G <= (D == 256 ? 64 : 128); }

cudaError_t keyscan_weights(const KeyScanParams& p, int D, int kind, cudaStream_t st) {
  switch (kind) {
    // the 16-bit kinds differ only in the instruction descriptor's type
    case KV_BF16:
    case KV_F16: return ks_weights_kind<KV_BF16>(p, D, st);
    case KV_I8: return ks_weights_kind<KV_I8>(p, D, st);
    case KV_I4: return ks_weights_kind<KV_I4>(p, D, st);
    case KV_F8: return ks_weights_kind<KV_F8>(p, D, st);
  }
  return cudaErrorInvalidValue;
}

cudaError_t keyscan_scores(const KeyScanParams& p, int D, cudaStream_t st) {
  if (D == 64) return ks_launch<64, SCAN_SCORES, KV_BF16>(p, st);
  if (D == 128) return ks_launch<128, SCAN_SCORES, KV_BF16>(p, st);
  if (D == 256) return ks_launch<256, SCAN_SCORES, KV_BF16>(p, st);
  return cudaErrorInvalidValue;
}

}  // namespace far
