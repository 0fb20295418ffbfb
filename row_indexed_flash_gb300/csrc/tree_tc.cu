// Attention of the nodes of a drafted tree on the 5th-generation tensor cores.
//
// The operation is that of tree.cu: every node of slice s sees the context's entries and, of the
// nodes at the list's end, itself and its ancestors.  The T * G query vectors of a KV head are few (8 to a
// few hundred) and the list is long, so the call is bound by reading K and V once: 4 T G flops for 4 bytes
// (16-bit pool) are below the tensor core's rate for up to some 280 query vectors.  Hence one CTA per
// SM, each with an equal share of all lists' tiles (tree.cuh), and every staged tile serves all query vectors.
//
// A tile is 64 entries.  A tile row is one (node, query head) pair of the KV head's group: S = Q K^T has up to
// 128 rows and a column per entry.  Two groups of four softmax warps (one thread a row) have two S and one O in
// tensor memory each, so a group's next product runs beside its softmax:
//   up to 128 query vectors: the groups take alternate tiles with the same Q; their sums are joined at a
//     unit's end (each thread reads its share of both O's columns)
//   more: each group has 128 query vectors of its own and takes every tile
//   D 256: one O fills half of the tensor memory, so there is one group
// Each group has an issuer of its own.  What a product costs its issuer is most of its time: the whole warp goes
// through the loop, so that operands stay in uniform registers, and one lane issues.  K and V are loaded by six warps
// (quantised pools: two): TMA boxes of 64 rows where the listed rows are one run, as pages are, else cp.async gathers
// into the same swizzled layout, whose rate goes by the number of warps.
// Measured on 16 sequences of 2k to 32k tokens in pages, 32/8 heads, 64 nodes (bf16, 768 MB): tiles of 128, one S a group
// and one issuer of one lane 313 us; tiles of 64 with two S 398, the issuer busy throughout; two issuers 324; converged
// warps 259; barriers that a poll has seen not waited for again, and asked side by side, 254; warps without a node idle,
// 249 to 252 (3.0 TB/s); one product for both S of a group 293, since it waits for both.  An f16 pool 256.  Codes, 24
// nodes: INT8 (389 MB) 166, INT4 175, E4M3 235.  4 x 16,384 shuffled bf16 rows, 16 nodes (270 MB): 75 (3.6 TB/s).
//
// The softmax keeps a reference per row that moves only when the maximum has grown by
// more than 2^8 (then O is rescaled in tensor memory); over 16-bit pools P goes over S as the pair rn(P), rn(P - rn(P)) of
// V's type, as in the decode kernel: one bf16 value (8 bits) would move outputs by up to 2^-9, one f16 value (11 bits) by up to
// 2^-12, and a token would be scored less exactly in a tree than decoded (f16 pool, 64 nodes: 217 us with one value, 256
// with the pair).
//
// Quantised pools (INT8, INT4, FP8 E4M3 codes with an fp16 scale per row and KV head; D 128):
//   codes      arrive in a ring of their own, their scales beside them
//   wideners   eight warps turn a tile's codes into 16-bit values in the products' layout: K in Q's type, V in f16,
//              exact in both (|code| <= 127, and every E4M3 value is an f16 and a bf16 value)
//   scales     the K scale multiplies the logit, the V scale the weight, which is then rounded once to f16 (11 bits, as in
//              quantised decode; a pair would cost 14 % over INT8, whose issue slots are scarce).  The references stand
//              2^E higher, 2^E being above every V scale of the unit's tiles so far, so weights stay within f16's range;
//              those of entries whose scale is within 2^-21 of the largest keep all 11 bits.
//
// Entries hidden by the tree have weight 0, but 0 * V is NaN where V is not finite.  Such values of nodes are
// therefore taken out of the staged V (by the softmax warps, of E4M3 codes by the wideners), and the rows that do see their
// node get them back at the end.  An infinity in the context of a 16-bit pool has a weight above 0, but the low part of that
// weight may be 0 or negative and a small one rounds to 0: a sum that came out NaN is looked up again at a unit's end.
//
// Every wait is bounded in time, as in the other tensor-core kernels.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <string.h>

#include <type_traits>

#include "kvread.cuh"
#include "tc.cuh"
#include "tmap.cuh"
#include "tree.cuh"
#include "widen.cuh"

namespace far {

namespace {

constexpr int kTtM = 128;                    // query vectors of a product = lanes of tensor memory
constexpr int kTtWords = kTreeMax / 32;      // words of a node's line: itself and its ancestors
constexpr int kTtWideners = 8;
// Weights that enter a product as f16 are taken 2^7 times as large: the lazy references bound them by 2^8,
// f16 by 2^16, and every power of two takes the smallest further from its subnormal range (steps of 2^-24).
constexpr float kTtLift = 7.f;

constexpr bool tt_quant(int kind) { return kind == KV_I8 || kind == KV_I4 || kind == KV_F8; }

template <int D, int KIND>
struct TreeShape {
  static constexpr bool QUANT = tt_quant(KIND);
  static constexpr int NG = D == 256 ? 1 : 2;          // softmax groups, and issuers
  static constexpr int BN = 64;                        // entries of a tile
  static constexpr int LOADERS = QUANT ? 2 : 6;
  static constexpr int NB = D / 64;                    // 64-column blocks of a row
  static constexpr int BLK = BN * 128;               // one block of a K or V tile
  static constexpr int TILE = BLK * NB;
  static constexpr int QBLK = kTtM * 128;
  static constexpr int QTILE = QBLK * NB;
  // stages of 16-bit tiles
  static constexpr int NSTK = QUANT ? 2 : D == 64 ? 8 : D == 128 ? 4 : 2;
  static constexpr int NSTV = QUANT ? 3 : NSTK;
  static constexpr int ROW = kv_row_bytes<KIND>(D);    // pool bytes of a row
  static constexpr int CODES = BN * ROW;             // code bytes of a tile and matrix
  static constexpr int NC = QUANT ? 49152 / (2 * CODES) : 0;   // code stages
  static constexpr int NSC = QUANT ? 8 : 0;                    // stages of scales
  // Slots for the notes of values that are not finite, a unit each in turn.  The end of unit u clears the slot that
  // unit u - 1 has read and unit u + NODD - 1 is to write.  Softmax warps, which write the notes of 16-bit pools, are at unit
  // u + 1 at most by then.  Wideners, which write those of codes, run ahead by the V stages: one at a unit w has the PV of
  // NSTV tiles before behind it, which is of unit w - NSTV or a later one (a unit has a tile at least), and the first
  // product of that into O waited for the end of the unit before.  So unit w's slot is clear by the end of w - NSTV - 1.
  static constexpr int NODD = QUANT ? NSTV + 2 : 3;
  static constexpr int NSMX = 4 * NG;                  // softmax warps
  static constexpr int W_LOAD = NSMX, W_MMA = NSMX + LOADERS, W_WIDE = W_MMA + NG;
  static constexpr int NWARP = W_WIDE + (QUANT ? kTtWideners : 0);
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = NG * QTILE;
  static constexpr int OFF_V = OFF_K + NSTK * TILE;
  static constexpr int OFF_C = OFF_V + NSTV * TILE;                  // [NC][K, V] codes
  static constexpr int OFF_CS = OFF_C + NC * 2 * CODES;              // [NC][K, V][64] fp16 scales
  static constexpr int OFF_SC = OFF_CS + NC * 2 * BN * 2;          // [NSC][c * s_k, s_v][64] fp32
  static constexpr int OFF_SE = OFF_SC + NSC * 2 * BN * 4;         // [NSC][2] E of the tile's halves
  static constexpr int OFF_BAR = OFF_SE + NSC * 2 * 4;
  // q_full, q_empty, o_free, drain [2], k_full, k_empty [NSTK], v_full, v_empty [NSTV], s_full, p_full, pv_done [2 groups][2],
  // comb [4], c_full, c_empty [NC]
  static constexpr int NBAR = 5 + 2 * NSTK + 2 * NSTV + 12 + 4 + 2 * NC;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;                // tensor memory's address, abort flag
  static constexpr int OFF_ODD = OFF_MISC + 16;                      // [NODD][kTtWords] nodes with a V not finite
  static constexpr int OFF_GATH = OFF_ODD + NODD * kTtWords * 4;      // [16] a stage was gathered: K, V
  static constexpr int OFF_IDX = OFF_GATH + 16 * 4;         // [loaders][64] rows of the tile a loader is on
  static constexpr int OFF_KIN = OFF_IDX + LOADERS * BN * 4;    // [NG][128][kTtWords] lines
  static constexpr int OFF_X = OFF_KIN + NG * kTtM * kTtWords * 4;   // [2 unit parities][2 groups][reference, sum][128]
  static constexpr int SMEM = OFF_X + 8 * kTtM * 4 + 1024;           // slack for 1024-byte alignment
  static constexpr uint32_t COL_S = 0, COL_O = 256;    // S b of group g at 64 (2 g + b), its O at COL_O + g * D
  static_assert(NG * D <= 256, "tensor memory");
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(OFF_SC % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
};

struct TreeTcParams {
  TreeParams a;
  int PT;       // nodes of a row tile
  int alt;      // 1: the groups take alternate tiles of one row tile, 0: a row tile each
  int tma_kv;   // 1: the K and V maps may be used
  int q_box;    // nodes of a Q box
};

// Drain wait: bounded in time, ignores the abort flag.
__device__ __forceinline__ void wait_drain(uint64_t* b, uint32_t parity) {
  const unsigned long long t0 = globaltimer();
  while (!mbar_try_wait(b, parity)) {
    if (globaltimer() - t0 > kWaitLimitNs) return;
  }
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
  return one != 0;
}
// The value of lane 0, which the compiler then knows to be the warp's.
__device__ __forceinline__ int of_warp(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Which of 32 entries from node u0 on a row sees (u0 < 0: entries before the nodes), kin: the row's words.
__device__ __forceinline__ uint32_t seen_bits(const uint32_t* kin, int u0) {
  if (u0 <= -32) return 0xffffffffu;
  if (u0 < 0) return (kin[0] << -u0) | ((1u << -u0) - 1u);
  const int w = u0 >> 5;
  if (w >= kTtWords) return 0u;
  const uint32_t hi = w + 1 < kTtWords ? kin[w + 1] : 0u;
  return __funnelshift_r(kin[w], hi, u0 & 31);
}

// Notes the line of node t of slice s (t < 0: none) in words of the calling
// thread's own.  Parents are smaller numbers, so the walk ends.
__device__ __forceinline__ void note_line(const TreeParams& p, int s, int t, uint32_t* kin) {
  for (int i = 0; i < kTtWords; ++i) kin[i] = 0u;
  while (t >= 0) {
    kin[t >> 5] |= 1u << (t & 31);
    const int q = __ldg(p.parent + (size_t)s * p.T + t);
    t = q < t ? q : -1;
  }
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}
// Codes to bf16 within 16-bit lanes, exact: a lane 0x43uu with uu < 128 is 128 + uu.  (Two instructions fewer for four INT4
// codes than by way of fp32, one fewer for INT8.)
// INT8: 128 + (the low seven bits) minus 128, or 256 for a negative code.
__device__ __forceinline__ uint2 codes_i8x4(uint32_t w) {
  const uint32_t a = __byte_perm(w, 0x43434343u, 0x4140u), b = __byte_perm(w, 0x43434343u, 0x4342u);
  return make_uint2(sub_bf16x2(a & 0xff7fff7fu, a & 0xff80ff80u), sub_bf16x2(b & 0xff7fff7fu, b & 0xff80ff80u));
}
// INT4 (element 2t in the low nibble of byte t): 128 + code + 8 minus 136.
__device__ __forceinline__ uint4 codes_i4x8(uint32_t w) {
  const uint32_t x = w ^ 0x88888888u, even = x & 0x0f0f0f0fu, odd = (x >> 4) & 0x0f0f0f0fu;
  const uint32_t p = __byte_perm(even, odd, 0x5140u), q = __byte_perm(even, odd, 0x7362u);   // elements 0-3, 4-7
  constexpr uint32_t k43 = 0x43434343u, k136 = 0x43084308u;
  return make_uint4(sub_bf16x2(__byte_perm(p, k43, 0x4140u), k136), sub_bf16x2(__byte_perm(p, k43, 0x4342u), k136),
                    sub_bf16x2(__byte_perm(q, k43, 0x4140u), k136), sub_bf16x2(__byte_perm(q, k43, 0x4342u), k136));
}
// Infinities among V's columns col .. col + 15 of KV head g, list positions lo .. hi - 1 of `rows`: bit k a +inf in column
// col + k, bit 16 + k a -inf, both bits for a NaN.  A whole warp calls it.
template <bool BF16>
__device__ __forceinline__ uint32_t odd_columns(const TreeParams& p, const int32_t* rows, int lo, int hi, int g, int col) {
  constexpr uint32_t INF = BF16 ? 0x7f80u : 0x7c00u;
  uint32_t found = 0;
#pragma unroll 1
  for (int pos = lo + (int)(threadIdx.x & 31); pos < hi; pos += 32) {
    const int row = __ldg(rows + pos);
    if (row < 0 || (long long)row >= p.R) continue;
    const uint4* at = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.v) + ((size_t)row * p.Hkv + g) * p.D + col);
    const uint4 a = __ldg(at), b = __ldg(at + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const uint32_t h = (w[k >> 1] >> (16 * (k & 1))) & 0xffffu, mag = h & 0x7fffu;
      if (mag >= INF) found |= mag > INF ? 0x10001u << k : h >> 15 ? 0x10000u << k : 1u << k;
    }
  }
  return __reduce_or_sync(0xffffffffu, found);
}
// 32 logits of a chunk: y = S * scale (quantised pools).
__device__ __forceinline__ void scale32(uint32_t (&sv)[32], const float* ksc) {
#pragma unroll
  for (int k = 0; k < 32; k += 4) {
    const float4 s4 = *reinterpret_cast<const float4*>(ksc + k);
    const float2 a = __fmul2_rn(make_float2(__uint_as_float(sv[k]), __uint_as_float(sv[k + 1])), make_float2(s4.x, s4.y));
    const float2 d = __fmul2_rn(make_float2(__uint_as_float(sv[k + 2]), __uint_as_float(sv[k + 3])), make_float2(s4.z, s4.w));
    sv[k] = __float_as_uint(a.x);
    sv[k + 1] = __float_as_uint(a.y);
    sv[k + 2] = __float_as_uint(d.x);
    sv[k + 3] = __float_as_uint(d.y);
  }
}
template <bool MAX>
__device__ __forceinline__ float extreme32(float x, const uint32_t (&sv)[32]) {
  float e[4] = {x, x, x, x};
  auto of = [](float a, float b) { return MAX ? fmaxf(a, b) : fminf(a, b); };
#pragma unroll
  for (int k = 0; k < 32; k += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      e[i] = of(e[i], of(__uint_as_float(sv[k + 2 * i]), __uint_as_float(sv[k + 2 * i + 1])));
  return of(of(e[0], e[1]), of(e[2], e[3]));
}

template <int D, int KIND, bool QBF16>
__global__ void __launch_bounds__(TreeShape<D, KIND>::NWARP * 32, 1)
    tree_tc_kernel(const __grid_constant__ TreeTcParams kp, const __grid_constant__ CUtensorMap tq,
                   const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
  using C = TreeShape<D, KIND>;
  constexpr bool QUANT = C::QUANT, PAIR = !QUANT, PBF16 = KIND == KV_BF16;   // P: two values, of bf16
  constexpr int BN = C::BN, NG = C::NG, LOADERS = C::LOADERS, NB = C::NB, NSTK = C::NSTK, NSTV = C::NSTV, NC = C::NC;
  const TreeParams& p = kp.a;
  const unsigned long long wait_ns = p.wait_ns;
  const float NEG_INF = __int_as_float(0xff800000);
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);   // stays a shared-memory address to the compiler
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  uint64_t* q_empty = q_full + 1;
  uint64_t* o_free = q_full + 2;    // the unit's sums have been read
  uint64_t* drain = q_full + 3;
  uint64_t* k_full = q_full + 5;
  uint64_t* k_empty = k_full + NSTK;
  uint64_t* v_full = k_empty + NSTK;
  uint64_t* v_empty = v_full + NSTV;
  uint64_t* s_full = v_empty + NSTV;   // [group][S]
  uint64_t* p_full = s_full + 4;
  uint64_t* pv_done = p_full + 4;
  uint64_t* comb = pv_done + 4;        // the two warps, one of each group, that share rows
  uint64_t* c_full = comb + 4;
  uint64_t* c_empty = c_full + NC;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::OFF_MISC + 4);
  uint32_t* odd = reinterpret_cast<uint32_t*>(sm + C::OFF_ODD);
  volatile int* gathered = reinterpret_cast<volatile int*>(sm + C::OFF_GATH);   // K stages, from 8 on V stages

  const int warp = of_warp(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int G = p.G, PT = kp.PT, alt = kp.alt;
  const int tiles_q = alt ? 1 : NG;                  // row tiles of a unit
  const int users = alt ? 1 : NG;                    // groups that a tile is for

  let_next_grid_start();
  tree_write_empty(p, threadIdx.x, C::NWARP * 32);
  const TreeWork work = tree_work(p);
  const int b = blockIdx.x;
  if (b >= work.shares || work.total == 0) return;
  const int lo = share_begin(work, b), hi = share_begin(work, b + 1);

  if (threadIdx.x == 0) {
    // a tile's loaders arrive with one lane each: asynchronously when its gathered copies land, or
    // plainly next to the TMA byte count
    constexpr int loads = LOADERS * 32;
    mbar_init(q_full, 1);
    mbar_init(q_empty, NG);
    mbar_init(o_free, C::NSMX);
    mbar_init(drain, 1);
    mbar_init(drain + 1, 1);
    for (int i = 0; i < NSTK; ++i) {
      mbar_init(k_full + i, QUANT ? kTtWideners / 2 : loads);
      mbar_init(k_empty + i, users);
    }
    for (int i = 0; i < NSTV; ++i) {
      mbar_init(v_full + i, QUANT ? kTtWideners / 2 : loads);
      mbar_init(v_empty + i, users);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 128);
      mbar_init(pv_done + i, 1);
      mbar_init(comb + i, 64);
    }
    if constexpr (QUANT) {
      for (int i = 0; i < NC; ++i) {
        mbar_init(c_full + i, loads);
        mbar_init(c_empty + i, kTtWideners);
      }
    }
    *abort_flag = 0;
    for (int i = 0; i < C::NODD * kTtWords; ++i) odd[i] = 0u;
    mbar_fence_init();
  }
  if (warp == C::W_MMA) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = of_warp(*tmem_holder);

  TreeUnit u = tree_unit(p, lo);
  // A role's registers (quantised pools, whose wideners leave a thread 96): a softmax thread holds 64 logits.
  // One instruction for each four warps, so loaders and MMA issuer take it together.
  if (warp >= C::W_LOAD && warp < C::W_WIDE) {
    if constexpr (QUANT) regs_release<72>();
    if (warp < C::W_MMA) {
      // -------------------------------------------------------------- loaders
      const int pi = warp - C::W_LOAD;
      const bool lead = pi == 0 && lane == 0;
      constexpr int E = BN / 32;               // entries a lane looks at
      constexpr int CPR = C::ROW / 16;         // 16-byte chunks of a row
      constexpr int RPI = 32 / CPR;            // rows of a warp's copy
      constexpr int NI = BN / RPI;             // copies of a tile
      constexpr int PER = (NI + LOADERS - 1) / LOADERS;   // of a loader: copies pi, pi + LOADERS, ...
      const int c = lane % CPR, er = lane / CPR;
      int32_t* idx = reinterpret_cast<int32_t*>(sm + C::OFF_IDX) + pi * BN;
      // TMA loads that may be in flight: bit st of K (of code stages), bit 16 + st of V, with their parities
      unsigned tma_pend = 0, tma_par = 0;
      int q_loads = 0;
      if (lead) {
        tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
      }
      bool ok = true;
      int jj = 0, ui = 0;
      for (int x = lo; ok && x < hi; u = tree_next(p, u), ++ui) {
        const int n_s = tree_len(p, u.s), t_lo = x - u.first, t_hi = min(u.tiles, hi - u.first);
        const int32_t* rows_u = p.kv_rows + (size_t)u.s * p.L;
        // two tiles ahead the list entries, one tile ahead the scales (loader 0), so that no load is waited for
        auto entries = [&](int t, int (&r)[E]) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int pos = t * BN + lane + 32 * e;
            r[e] = t < t_hi && pos < n_s ? __ldg(rows_u + pos) : -1;
          }
        };
        auto clip = [&](int (&r)[E]) {
#pragma unroll
          for (int e = 0; e < E; ++e)
            if ((long long)r[e] >= p.R) r[e] = -1;
        };
        auto scales = [&](const int (&r)[E], uint16_t (&ks)[E], uint16_t (&vs)[E]) {
          if (!QUANT || pi != 0) return;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const size_t o = r[e] >= 0 ? ((size_t)(r[e] >> 6) * p.Hkv + u.g) * kPage + (r[e] & 63) : 0;
            ks[e] = r[e] >= 0 ? __ldg(p.k_scale + o) : (uint16_t)0;
            vs[e] = r[e] >= 0 ? __ldg(p.v_scale + o) : (uint16_t)0;
          }
        };
        int rows[E], nxt[E];
        uint16_t ks[E] = {}, vs[E] = {};
        entries(t_lo, rows);
        entries(t_lo + 1, nxt);
        clip(rows);
        scales(rows, ks, vs);
        if (lead) {
          ok = mbar_wait(q_empty, (ui & 1) ^ 1, abort_flag, wait_ns);
          if (ok) {
            mbar_arrive_expect_tx(q_full, (uint32_t)tiles_q * NB * (uint32_t)(kp.q_box * G) * 128u);
            for (int qt = 0; qt < tiles_q; ++qt)
              for (int h = 0; h < NB; ++h)
                tma_load_3d(sm + C::OFF_Q + qt * C::QTILE + h * C::QBLK, &tq, h * 64, u.g * G,
                            u.s * p.T + (u.rt * tiles_q + qt) * PT, q_full);
            ++q_loads;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        for (int t = t_lo; ok && t < t_hi; ++t, ++jj) {
          int later[E];
          entries(t + 2, later);
          clip(nxt);
          uint16_t nks[E] = {}, nvs[E] = {};
          scales(nxt, nks, nvs);
          int run[E / 2];   // the first row of each 64
          bool contig = kp.tma_kv != 0;
#pragma unroll
          for (int h = 0; h < E / 2; ++h) {
            run[h] = __shfl_sync(0xffffffffu, rows[2 * h], 0);
            contig = contig && run[h] >= 0 && rows[2 * h] == run[h] + lane && rows[2 * h + 1] == run[h] + 32 + lane;
          }
          contig = __all_sync(0xffffffffu, contig);
          if (!contig) {
            __syncwarp();
#pragma unroll
            for (int e = 0; e < E; ++e) idx[lane + 32 * e] = rows[e];
            __syncwarp();
          }
          // this warp's share of the gathered rows, 16-byte chunk c of row pi * RPI + er and so on; the rows
          // are read before any copy goes out, which the compiler would not move them past
          int mine[PER];
          if (!contig) {
#pragma unroll
            for (int i = 0; i < PER; ++i) mine[i] = idx[min(pi + LOADERS * i, NI - 1) * RPI + er];
          }
          auto gather = [&](const void* src, auto at) {
            const char* from = static_cast<const char*>(src) + (size_t)u.g * C::ROW + c * 16;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
              if (NI % LOADERS && pi + LOADERS * i >= NI) break;
              const bool there = mine[i] >= 0;
              cp_async16(at((pi + LOADERS * i) * RPI + er), from + (size_t)(there ? mine[i] : 0) * p.Hkv * C::ROW, there);
            }
          };
          if constexpr (QUANT) {
            const int st = jj % (NC ? NC : 1), ph = (jj / (NC ? NC : 1)) & 1;
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(c_empty + st, ph ^ 1, abort_flag, wait_ns)))) break;
            if (pi == 0) {
              uint16_t* cs = reinterpret_cast<uint16_t*>(sm + C::OFF_CS) + st * 2 * BN;
#pragma unroll
              for (int e = 0; e < E; ++e) {
                cs[lane + 32 * e] = ks[e];
                cs[BN + lane + 32 * e] = vs[e];
              }
            }
            unsigned char* dst = sm + C::OFF_C + st * 2 * C::CODES;
            if (lead) tma_pend &= ~(1u << st);
            if (contig) {
              if (lead) {
                mbar_arrive_expect_tx(c_full + st, 2 * C::CODES);
                tma_load_3d(dst, &tk, 0, u.g, run[0], c_full + st);
                tma_load_3d(dst + C::CODES, &tv, 0, u.g, run[0], c_full + st);
                tma_pend |= 1u << st;
                tma_par = (tma_par & ~(1u << st)) | ((unsigned)ph << st);
              } else {
                mbar_arrive(c_full + st);
              }
            } else {
              gather(p.k, [&](int e) { return dst + e * C::ROW + c * 16; });
              gather(p.v, [&](int e) { return dst + C::CODES + e * C::ROW + c * 16; });
              if (pi == 0) __threadfence_block();   // the scales before the copies' own arrival
              cp_async_mbar_arrive_noinc(c_full + st);
            }
          } else {
            auto load = [&](unsigned char* dst, const void* map, const void* src, uint64_t* full, int ph, int bit) {
              if (lead) {
                tma_pend &= ~(1u << bit);
                gathered[(bit & 15) + (bit >> 4) * 8] = !contig;
              }
              if (contig) {
                if (lead) {
                  mbar_arrive_expect_tx(full, C::TILE);
#pragma unroll
                  for (int h = 0; h < E / 2; ++h)
#pragma unroll
                    for (int k = 0; k < NB; ++k) tma_load_3d(dst + k * C::BLK + h * 64 * 128, map, k * 64, u.g, run[h], full);
                  tma_pend |= 1u << bit;
                  tma_par = (tma_par & ~(1u << bit)) | ((unsigned)ph << bit);
                } else {
                  mbar_arrive(full);
                }
              } else {
                gather(src, [&](int e) { return dst + (c >> 3) * C::BLK + e * 128 + (((c & 7) ^ (e & 7)) << 4); });
                if (lead) __threadfence_block();   // the note before the copies' own arrival
                cp_async_mbar_arrive_noinc(full);
              }
            };
            const int sk = jj % NSTK, pk = (jj / NSTK) & 1, sv = jj % NSTV, pv = (jj / NSTV) & 1;
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(k_empty + sk, pk ^ 1, abort_flag, wait_ns)))) break;
            load(sm + C::OFF_K + sk * C::TILE, &tk, p.k, k_full + sk, pk, sk);
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(v_empty + sv, pv ^ 1, abort_flag, wait_ns)))) break;
            load(sm + C::OFF_V + sv * C::TILE, &tv, p.v, v_full + sv, pv, 16 + sv);
          }
#pragma unroll
          for (int e = 0; e < E; ++e) {
            rows[e] = nxt[e];
            nxt[e] = later[e];
            ks[e] = nks[e];
            vs[e] = nvs[e];
          }
        }
        x = u.first + t_hi;
      }
      cp_async_wait_all();
      // bulk copies still in flight must land before the CTA can exit, whether or not a wait has run out
      if (lead) {
        if (q_loads) wait_drain(q_full, (q_loads - 1) & 1);
        for (int st = 0; st < 16; ++st) {
          if ((tma_pend >> st) & 1u) wait_drain((QUANT ? c_full : k_full) + st, (tma_par >> st) & 1u);
          if ((tma_pend >> (16 + st)) & 1u) wait_drain(v_full + st, (tma_par >> (16 + st)) & 1u);
        }
      }
    } else {
      // ---------------------------------------------------------- MMA issuers
      // One for each group, so that a group's products stay in order: a QK may go out once one of its S is
      // free (its PV has been issued) and the K stage is there, a PV once its P is written and its V stage there.
      const int g = warp - C::W_MMA;
      const uint32_t id_qk = make_idesc_f16(kTtM, BN, QBF16, false);
      const uint32_t id_pv = make_idesc_f16(kTtM, D, PBF16, true);
      const uint64_t dQ = sdesc_at(sdesc_sw128(smem_u32(sm + C::OFF_Q), 16, 1024), alt ? 0 : g * C::QTILE);
      const uint64_t dK = sdesc_sw128(smem_u32(sm + C::OFF_K), 16, 1024);
      const uint64_t dV = sdesc_sw128(smem_u32(sm + C::OFF_V), C::BLK, 1024);
      const uint32_t tS0 = tbase + C::COL_S + g * 2 * BN, tOg = tbase + C::COL_O + g * D;
      const int step = alt ? 2 : 1;
      // The whole warp goes through the loop and one lane issues: the operands then stay
      // in uniform registers (a loop of one lane moved them there for every product)
      auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
      bool ok = true;
      int jj0 = 0, ui = 0, cq = 0, cp = 0;   // cq, cp: the group's tiles so far whose QK, PV have been issued
      for (int x = lo; ok && x < hi; u = tree_next(p, u), ++ui) {
        const int t_lo = x - u.first, t_hi = min(u.tiles, hi - u.first), n = of_warp(t_hi - t_lo);
        const int start = alt ? (g - jj0) & 1 : 0;
        int nq = start, np = start;   // next tile of QK, PV
        // with no tile of its own too: a phase skipped could be mistaken for the one after
        ok = all(mbar_wait(q_full, ui & 1, abort_flag, wait_ns));
        if (start >= n && lane == 0) mbar_arrive(q_empty);
        while (ok && np < n) {
          const int jq = jj0 + nq, sk = jq % NSTK, pk = (jq / NSTK) & 1;
          const int jp = jj0 + np, sv = jp % NSTV, sp = cp & 1;
          const bool may_qk = nq < n && cq - cp < 2, may_pv = np < nq;
          // wait where only one can be next, else take what comes first: the barriers are asked side by side, as an
          // answer takes 100 clocks
          bool qk = may_qk, pv = may_pv;
          uint64_t* pb = p_full + 2 * g + sp;
          const uint32_t pp = (cp >> 1) & 1, vp = (jp / NSTV) & 1;
          const bool fresh = np == start && ui > 0;   // O begins anew: the unit before has been read
          if (may_qk && may_pv) {
            unsigned long long t_idle = 0;
            while (ok) {
              const bool k_in = mbar_test_wait(k_full + sk, pk);
              const bool p_in = mbar_test_wait(pb, pp), v_in = mbar_test_wait(v_full + sv, vp);
              const bool o_in = !fresh || mbar_test_wait(o_free, (ui - 1) & 1);
              qk = all(k_in);
              pv = all(p_in && v_in && o_in);
              if (qk || pv) break;
              bool late = false;
              if (t_idle == 0) t_idle = globaltimer();
              else late = *abort_flag || globaltimer() - t_idle > wait_ns;
              if (late) *abort_flag = 1;
              ok = all(!late);
            }
          } else if (may_qk) {
            ok = all(mbar_wait(k_full + sk, pk, abort_flag, wait_ns));
          } else {
            ok = all(mbar_wait(pb, pp, abort_flag, wait_ns) && mbar_wait(v_full + sv, vp, abort_flag, wait_ns) &&
                     (!fresh || mbar_wait(o_free, (ui - 1) & 1, abort_flag, wait_ns)));
          }
          if (!ok) break;
          if (pv) {
            tc_fence_after();
            if (!QUANT && of_warp(gathered[8 + sv])) fence_proxy_async_smem();
            const uint32_t a = tS0 + sp * BN;
            const uint64_t v = sdesc_at(dV, sv * C::TILE);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < BN / 16; ++kk) {
                // P of entries 16kk .. 16kk+15 at column 16kk; its low part at 16kk + 8
                const uint64_t vd = sdesc_at(v, kk * 2048);
                mma_ts(tOg, a + kk * 16, vd, id_pv, np != start || kk > 0);
                if constexpr (PAIR) mma_ts(tOg, a + kk * 16 + 8, vd, id_pv, 1);
              }
              tc_commit(v_empty + sv);
              tc_commit(pv_done + 2 * g + sp);
            }
            __syncwarp();
            np += step;
            ++cp;
          }
          if (qk) {
            tc_fence_after();
            if (!QUANT && of_warp(gathered[sk])) fence_proxy_async_smem();
            const uint32_t d = tS0 + (cq & 1) * BN;
            const uint64_t k = sdesc_at(dK, sk * C::TILE);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                mma_ss(d, sdesc_at(dQ, (kk >> 2) * C::QBLK + (kk & 3) * 32),
                       sdesc_at(k, (kk >> 2) * C::BLK + (kk & 3) * 32), id_qk, kk > 0);
              tc_commit(s_full + 2 * g + (cq & 1));
              tc_commit(k_empty + sk);
              if (nq + step >= n) tc_commit(q_empty);
            }
            __syncwarp();
            nq += step;
            ++cq;
          }
        }
        jj0 += n;
        x = u.first + t_hi;
      }
      if (elect_one()) tc_commit(drain + g);
      __syncwarp();
      wait_drain(drain + g, 0);
    }
  } else if (QUANT && warp >= C::W_WIDE) {
    // ------------------------------------------------------------- wideners
    if constexpr (QUANT) {
      regs_release<72>();
      // four warps for K and four for V: neither waits for the other's stage
      const bool values = warp >= C::W_WIDE + kTtWideners / 2;
      const int tid = (warp - C::W_WIDE) % (kTtWideners / 2) * 32 + lane;
      constexpr int CPR = C::ROW / 16, CHUNKS = BN * CPR, NT = kTtWideners / 2 * 32;
      bool ok = true;
      int jj = 0, ui = 0;
      for (int x = lo; ok && x < hi; u = tree_next(p, u), ++ui) {
        const int t_lo = x - u.first, t_hi = min(u.tiles, hi - u.first);
        int base = 0;
        if constexpr (KIND == KV_F8) base = tree_len(p, u.s) - tree_nodes(p, u.s);
        uint32_t* odd_u = odd + ui % C::NODD * kTtWords;
        for (int t = t_lo; t < t_hi; ++t, ++jj) {
          const int sc = jj % NC, sk = jj % NSTK, sv = jj % NSTV;
          unsigned char* codes = sm + C::OFF_C + sc * 2 * C::CODES;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(c_full + sc, (jj / NC) & 1, abort_flag, wait_ns) &&
                                                 (values ? mbar_wait(v_empty + sv, ((jj / NSTV) & 1) ^ 1, abort_flag, wait_ns)
                                                         : mbar_wait(k_empty + sk, ((jj / NSTK) & 1) ^ 1, abort_flag, wait_ns)))))
            break;
          // 16-byte chunks of codes to 32 or 64 bytes of 16-bit values of their row
          auto widen = [&](const unsigned char* src, unsigned char* tile, auto bf16_t) {
            constexpr bool bf16 = decltype(bf16_t)::value;
#pragma unroll
            for (int f0 = 0; f0 < CHUNKS; f0 += NT) {
              const int f = f0 + tid;
              const int e = f / CPR, cc = f % CPR;
              uint4 w = *reinterpret_cast<const uint4*>(src + f * 16);
              if constexpr (KIND == KV_F8) {
                const int k = t * BN + e - base;
                if (values && k >= 0) {
                  // NaN codes of a node leave V
                  uint32_t ws[4] = {w.x, w.y, w.z, w.w}, any = 0;
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const uint32_t hit = ((ws[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                    any |= hit;
                    ws[i] &= ~((hit >> 7) * 0xffu);
                  }
                  if (any) {
                    if (k < kTreeMax) atomicOr(odd_u + (k >> 5), 1u << (k & 31));
                    w = make_uint4(ws[0], ws[1], ws[2], ws[3]);
                  }
                }
              }
              auto put = [&](int unit, uint4 v) {   // 16-byte unit of the row
                *reinterpret_cast<uint4*>(tile + (unit >> 3) * C::BLK + e * 128 + (((unit & 7) ^ (e & 7)) << 4)) = v;
              };
              // Lanes of the row's two halves store units of unlike parity at a time: those of equal parity of two
              // 64-column blocks lie in the same banks (INT8 172 us without, 167 with; E4M3 and INT4 gain nothing).
              const int far_half = KIND == KV_I8 && cc >= CPR / 2;
              if constexpr (KIND == KV_I4) {
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) put(4 * cc + i, bf16 ? codes_i4x8(ws[i]) : widen_i4x8(ws[i], false));
              } else {
                const uint32_t ws[4] = {far_half ? w.z : w.x, far_half ? w.w : w.y, far_half ? w.x : w.z, far_half ? w.y : w.w};
                uint2 o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  if constexpr (KIND == KV_I8) {
                    o[i] = bf16 ? codes_i8x4(ws[i]) : widen_i8x4(ws[i], false);
                  } else {
                    o[i] = widen_e4m3x4(ws[i]);
                    if constexpr (bf16) {
                      const float2 a = f16x2_to_f2(o[i].x), d = f16x2_to_f2(o[i].y);
                      o[i] = make_uint2(pack2h(a.x, a.y, true), pack2h(d.x, d.y, true));
                    }
                  }
                }
                put((2 * cc) ^ far_half, make_uint4(o[0].x, o[0].y, o[1].x, o[1].y));
                put((2 * cc + 1) ^ far_half, make_uint4(o[2].x, o[2].y, o[3].x, o[3].y));
              }
            }
          };
          if (values) {
            widen(codes + C::CODES, sm + C::OFF_V + sv * C::TILE, std::false_type{});
          } else {
            // Scales: the place's last reader was the softmax of eight tiles ago.  It has ended: the K stages of this tile
            // and the one before waited for the products of two and three tiles ago, and each of those took an S that
            // its group's softmax of four tiles earlier (two, where both groups take every tile) had done with.
            float* sc_f = reinterpret_cast<float*>(sm + C::OFF_SC) + jj % C::NSC * 2 * BN;
            const uint32_t h = reinterpret_cast<const uint16_t*>(sm + C::OFF_CS)[sc * 2 * BN + tid];
            static_assert(NT == 2 * BN, "a scale a thread");
            sc_f[tid] = __half2float(__ushort_as_half((unsigned short)h)) * (tid < BN ? p.qscale : 1.f);
            // 2^E above the finite scales: from the largest exponent
            const uint32_t mag = h & 0x7fffu, top = __reduce_max_sync(0xffffffffu, mag < 0x7c00u ? mag : 0u);
            if (lane == 0 && tid >= BN)
              reinterpret_cast<float*>(sm + C::OFF_SE)[jj % C::NSC * 2 + (tid - BN) / 32] = (float)((int)(top >> 10) - 14);
            widen(codes, sm + C::OFF_K + sk * C::TILE, std::integral_constant<bool, QBF16>{});
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(values ? v_full + sv : k_full + sk);
            mbar_arrive(c_empty + sc);
          }
        }
        x = u.first + t_hi;
      }
    }
  } else {
    // -------------------------------------------------------------- softmax
    if constexpr (QUANT) regs_acquire<128>();
    const int grp = warp >> 2, quad = warp & 3;
    const int m = quad * 32 + lane;
    const uint32_t lane_sel = (uint32_t)(quad * 32) << 16;
    const uint32_t tO = tbase + lane_sel + C::COL_O + grp * D;
    float* xs = reinterpret_cast<float*>(sm + C::OFF_X);   // [parity][group][reference, sum][row]
    uint32_t* kin = reinterpret_cast<uint32_t*>(sm + C::OFF_KIN) + (grp * kTtM + m) * kTtWords;
    // 16-bit pools: c = scale * log2(e) is applied to S in the exponent; a zero scale is replaced by the smallest
    // normal float, which leaves every logit 0 to within 2^-100 while a hidden entry's infinite fill still
    // maps to -inf.  Quantised pools: c is in the K scales already.
    const float c = QUANT ? 1.f : p.qscale == 0.f ? 1.17549435e-38f : p.qscale;
    const uint32_t fill = c > 0.f ? 0xff800000u : 0x7f800000u;
    bool ok = true;
    int jj0 = 0, ui = 0, done = 0;   // done: tiles of this group
    for (int x = lo; ok && x < hi; u = tree_next(p, u), ++ui) {
      const int n_s = tree_len(p, u.s), nn = tree_nodes(p, u.s), base = n_s - nn;
      const int t_lo = x - u.first, t_hi = min(u.tiles, hi - u.first), n = t_hi - t_lo;
      const int node = (u.rt * tiles_q + (alt ? 0 : grp)) * PT + m / G;
      const bool row_ok = m < PT * G && node < p.T;
      const bool live = row_ok && node < nn;
      // A warp without a node keeps the products' steps alone (16 sequences of 33 to 64 nodes: 254 us without, 249 with).
      // Over codes the wideners set the pace, and the branch costs (64 nodes 262 us without, 264 with).
      const bool idle = !QUANT && !__any_sync(0xffffffffu, live);
      const int32_t* rows_u = p.kv_rows + (size_t)u.s * p.L;
      const int step = alt ? 2 : 1, start = alt ? (grp - jj0) & 1 : 0;
      uint32_t* odd_u = odd + ui % C::NODD * kTtWords;
      // list entries of the group's next tile, loaded a tile ahead
      int nxt[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int pos = (t_lo + start) * BN + lane + 32 * q;
        nxt[q] = start < n && pos < n_s ? __ldg(rows_u + pos) : -1;
      }
      const bool tail = t_hi * BN > base;   // this share of the unit holds nodes
      if (tail) note_line(p, u.s, live ? node : -1, kin);
      // weights are exp2(logit - ref), sums relative to it.  shift: how far the reference stands above the largest
      // logit when it is set (-7 for f16 weights; above V scales for quantised pools)
      float ref = NEG_INF, l = 0.f;
      float shift = PBF16 ? 0.f : QUANT ? -14.f - kTtLift : -kTtLift;
      for (int j = start; j < n; j += step, ++done) {
        const int jb = (t_lo + j) * BN;   // list position of the tile's first entry
        uint32_t bits[2];
        // a row without a node has an empty line: in tiles with nodes it sees the context alone (its sums are dropped)
        bool masked = false;
        const bool nodes_here = jb + BN > base;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          bits[q] = __ballot_sync(0xffffffffu, nxt[q] >= 0 && (long long)nxt[q] < p.R);
          const int pos = jb + step * BN + lane + 32 * q;
          nxt[q] = j + step < n && pos < n_s ? __ldg(rows_u + pos) : -1;
          if (nodes_here && !idle) bits[q] &= seen_bits(kin, jb + 32 * q - base);
          masked = masked || bits[q] != 0xffffffffu;
        }
        const int sb = 2 * grp + (done & 1);
        const uint32_t tS = tbase + lane_sel + C::COL_S + sb * BN;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(s_full + sb, (done >> 1) & 1, abort_flag, wait_ns)))) break;
        tc_fence_after();
        if (!idle) {
          const int sc = QUANT ? (jj0 + j) % (QUANT ? C::NSC : 1) : 0;
          const float* ksc = reinterpret_cast<const float*>(sm + C::OFF_SC) + sc * 2 * BN;
          uint32_t sv[2][32];
          tmem_ld32_nowait(tS, sv[0]);
          tmem_ld32_nowait(tS + 32, sv[1]);
          tmem_wait_ld_tied(sv[0]);
          tmem_wait_ld_tied(sv[1]);
          float top = __uint_as_float(fill);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if constexpr (QUANT) scale32(sv[q], ksc + 32 * q);
            if (masked) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!((bits[q] >> k) & 1u)) sv[q][k] = fill;
            }
            if (QUANT || c > 0.f) top = extreme32<true>(top, sv[q]);
            else top = extreme32<false>(top, sv[q]);
          }
          if constexpr (QUANT) {
            const float* se = reinterpret_cast<const float*>(sm + C::OFF_SE) + sc * 2;
            shift = fmaxf(shift, fmaxf(se[0], se[1]) - kTtLift);
          }
          const float want = __float_as_uint(top) == fill ? NEG_INF : top * c + shift;
          const bool need = want > ref + 8.f;
          if (__any_sync(0xffffffffu, need)) {
            // rare: move the reference and rescale O in place, once the group's last PV has completed
            const float alpha = need ? fast_ex2(ref - want) : 1.f;
            if (need) {
              l *= alpha;
              ref = want;
            }
            if (j != start) {
              const int before = 2 * grp + ((done - 1) & 1);
              ok = __all_sync(0xffffffffu, mbar_wait(pv_done + before, ((done - 1) >> 1) & 1, abort_flag, wait_ns));
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int c4 = 0; c4 < D; c4 += 16) {
                uint32_t r[16];
                tmem_ld16(tO + c4, r);
#pragma unroll
                for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * alpha);
                tmem_st16(tO + c4, r);
              }
            }
          }
          // P over S, 16 entries at a time: (the high parts) to the first 8 columns, low parts to the others
          const float nm = ref == NEG_INF ? 0.f : -ref;
          const float2 c2 = make_float2(c, c), nm2 = make_float2(nm, nm);
          float2 acc = make_float2(0.f, 0.f);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int o = 0; o < 4; ++o) {
              uint32_t w[8];
              float4 v4[2];   // V scales of these entries
              if constexpr (QUANT) {
                v4[0] = *reinterpret_cast<const float4*>(ksc + BN + 32 * q + 8 * o);
                v4[1] = *reinterpret_cast<const float4*>(ksc + BN + 32 * q + 8 * o + 4);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int i = 8 * o + 2 * k;
                const float2 s2 = make_float2(__uint_as_float(sv[q][i]), __uint_as_float(sv[q][i + 1]));
                const float2 t = QUANT ? __fadd2_rn(s2, nm2) : __ffma2_rn(s2, c2, nm2);
                float2 pr = make_float2(fast_ex2(t.x), fast_ex2(t.y));
                acc = __fadd2_rn(acc, pr);
                if constexpr (QUANT) {
                  const float4& f4 = v4[k >> 1];
                  pr = __fmul2_rn(pr, k & 1 ? make_float2(f4.z, f4.w) : make_float2(f4.x, f4.y));
                  if (masked) {   // a hidden entry's scale may be anything
                    pr.x = (bits[q] >> i) & 1u ? pr.x : 0.f;
                    pr.y = (bits[q] >> (i + 1)) & 1u ? pr.y : 0.f;
                  }
                }
                const uint32_t h = pack2h(pr.x, pr.y, PBF16);
                w[k] = h;
                if constexpr (PAIR) {
                  const float2 hi =
                      PBF16 ? make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u)) : f16x2_to_f2(h);
                  const float2 rem = __fadd2_rn(pr, make_float2(-hi.x, -hi.y));
                  w[4 + k] = pack2h(rem.x, rem.y, PBF16);
                }
              }
              const uint32_t col = tS + (2 * q + (o >> 1)) * 16 + (o & 1) * 4;
              tmem_st4_nowait(col, w[0], w[1], w[2], w[3]);
              if constexpr (PAIR) tmem_st4_nowait(col + 8, w[4], w[5], w[6], w[7]);
            }
          }
          l += acc.x + acc.y;
          tmem_wait_st();
        }
        if (!QUANT && nodes_here) {
          // values of nodes that are not finite leave the staged V
          const int st = (jj0 + j) % NSTV;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(v_full + st, ((jj0 + j) / NSTV) & 1, abort_flag, wait_ns)))) break;
          unsigned char* vt = sm + C::OFF_V + st * C::TILE;
          constexpr uint32_t ADD = PBF16 ? 0x00800080u : 0x04000400u;   // carries a magnitude that is not finite into bit 15
          for (int f = m; f < C::TILE / 16; f += 128) {
            uint4* at = reinterpret_cast<uint4*>(vt) + f;
            const int k = jb + (f * 16 % C::BLK) / 128 - base;
            if (k < 0) continue;
            const uint4 v = *at;
            uint32_t w[4] = {v.x, v.y, v.z, v.w}, any = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t hit = ((w[i] & 0x7fff7fffu) + ADD) & 0x80008000u;
              any |= hit;
              w[i] &= ~((hit >> 15) * 0xffffu);
            }
            if (any) {
              if (k < kTreeMax) atomicOr(odd_u + (k >> 5), 1u << (k & 31));
              __threadfence_block();
              *at = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(p_full + sb);
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;

      // the unit's sums
      float* x0 = xs + (ui & 1) * 4 * kTtM + m;
      bool had[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) had[g] = g < NG && (alt ? ((g - jj0) & 1) < n : true);
      if (alt) {
        x0[(grp * 2) * kTtM] = ref;
        x0[(grp * 2 + 1) * kTtM] = l;
        mbar_arrive(comb + quad);
        ok = mbar_wait(comb + quad, ui & 1, abort_flag, wait_ns);
      }
      // the last PV of each group that had tiles: the number of its last tile among the group's
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (!had[g] || (!alt && g != grp)) continue;
        const int last = (alt ? (jj0 + n + 1 - g) >> 1 : jj0 + n) - 1;
        ok = ok && mbar_wait(pv_done + 2 * g + (last & 1), (last >> 1) & 1, abort_flag, wait_ns);
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      // This wait says that the unit before is behind every warp (its sums were read before this one's first
      // product into O went out): its notes make room for those of unit ui + NODD - 1, whose writers wait for this end.
      if (threadIdx.x < kTtWords) odd[(ui + C::NODD - 1) % C::NODD * kTtWords + threadIdx.x] = 0u;
      tc_fence_after();
      // this thread's columns: with alternate tiles half of both groups' sums, joined at the larger
      // reference; else all of its own
      float a0 = 1.f, a1 = 0.f, lt = l;
      if (alt) {
        const float m0 = x0[0], m1 = x0[2 * kTtM];
        ref = fmaxf(m0, m1);
        const float z = ref == NEG_INF ? 0.f : ref;
        a0 = fast_ex2(m0 - z);
        a1 = fast_ex2(m1 - z);
        lt = x0[kTtM] * a0 + x0[3 * kTtM] * a1;
      }
      if (!live) {
        lt = 0.f;
        ref = NEG_INF;
      }
      const bool whole = t_lo == 0 && t_hi == u.tiles;
      const bool none = !live || (whole && lt == 0.f);
      const float inv = whole ? 1.f / lt : 1.f;
      const int span = alt ? D / 2 : D, col0 = alt ? grp * span : 0;
      const size_t oi = ((size_t)u.s * p.T + node) * p.Hq + u.g * G + m % G;
      const size_t pi = (size_t)(2 * b + (x == lo ? 0 : 1)) * p.rows + (alt ? 0 : grp) * PT * G + m;
      uint32_t any_odd = 0;
      if (tail) {
#pragma unroll
        for (int i = 0; i < kTtWords; ++i) any_odd |= reinterpret_cast<volatile uint32_t*>(odd_u)[i];
      }
#pragma unroll 1
      for (int cc = 0; cc < span; cc += 16) {
        const int col = col0 + cc;
        uint32_t r[16];
        float y[16];
        if (alt) {
#pragma unroll
          for (int k = 0; k < 16; ++k) y[k] = 0.f;
          if (had[0]) {
            tmem_ld16(tbase + lane_sel + C::COL_O + col, r);
#pragma unroll
            for (int k = 0; k < 16; ++k) y[k] = __uint_as_float(r[k]) * a0;
          }
          if (had[1]) {
            tmem_ld16(tbase + lane_sel + C::COL_O + (NG - 1) * D + col, r);
#pragma unroll
            for (int k = 0; k < 16; ++k) y[k] = fmaf(__uint_as_float(r[k]), a1, y[k]);
          }
        } else {
          tmem_ld16(tO + col, r);
#pragma unroll
          for (int k = 0; k < 16; ++k) y[k] = __uint_as_float(r[k]);
        }
        if constexpr (!QUANT) {
          // a sum that is NaN though the weights are not: infinities of the context, which every node sees
          bool nan = false;
#pragma unroll
          for (int k = 0; k < 16; ++k) nan = nan || y[k] != y[k];
          nan = nan && live && lt == lt;
          if (__any_sync(0xffffffffu, nan)) {
            const uint32_t found = odd_columns<PBF16>(p, rows_u, t_lo * BN, min(min(t_hi * BN, n_s), base), u.g, col);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const uint32_t signs = (found >> k) & 0x10001u;
              if (nan && y[k] != y[k] && (signs == 1u || signs == 0x10000u))
                y[k] = __uint_as_float(signs == 1u ? 0x7f800000u : 0xff800000u);
            }
          }
        }
        if (!row_ok) continue;
        if (any_odd) {
          // values that were taken out, for the rows that see their node
          for (int i = 0; i < kTtWords; ++i)
            for (uint32_t w = odd_u[i] & kin[i]; w; w &= w - 1) {
              const int k = i * 32 + __ffs(w) - 1, pos = base + k;
              const int row = pos >= 0 && pos < n_s ? __ldg(rows_u + pos) : -1;
              if (row < 0 || (long long)row >= p.R) continue;
              const size_t at = ((size_t)row * p.Hkv + u.g) * D + col;
#pragma unroll
              for (int t = 0; t < 16; ++t) {
                if constexpr (QUANT) {
                  if (KIND == KV_F8 && (__ldg(static_cast<const uint8_t*>(p.v) + at + t) & 0x7f) == 0x7f)
                    y[t] = __int_as_float(0x7fc00000);
                } else {
                  const uint32_t h = __ldg(static_cast<const uint16_t*>(p.v) + at + t);
                  const float f = PBF16 ? __uint_as_float(h << 16) : __half2float(__ushort_as_half((unsigned short)h));
                  if (!isfinite(f)) y[t] += f;
                }
              }
            }
        }
        if (whole || none) {
#pragma unroll
          for (int k = 0; k < 16; ++k) y[k] = none ? 0.f : y[k] * inv;
        }
        if (!whole || p.out_dtype == FA_F32) {
          float4* o4 = reinterpret_cast<float4*>(whole ? static_cast<float*>(p.out) + oi * D + col : p.part_o + pi * D + col);
#pragma unroll
          for (int k = 0; k < 4; ++k) o4[k] = make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
        } else {
          const bool ob = p.out_dtype == FA_BF16;
          uint4* o4 = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + oi * D + col);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            o4[k] = make_uint4(pack2h(y[8 * k], y[8 * k + 1], ob), pack2h(y[8 * k + 2], y[8 * k + 3], ob),
                               pack2h(y[8 * k + 4], y[8 * k + 5], ob), pack2h(y[8 * k + 6], y[8 * k + 7], ob));
        }
      }
      if (row_ok && (!alt || grp == 0)) {
        if (whole) {
          if (p.lse) p.lse[oi] = lt != 0.f ? (ref + __log2f(lt)) * kLn2 : NEG_INF;
        } else {
          *reinterpret_cast<float2*>(p.part_ml + pi * 2) = make_float2(ref, lt);
        }
      }
      // O may be written again
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
      jj0 += n;
      x = u.first + t_hi;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::W_MMA) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
  if (threadIdx.x == 0 && *abort_flag && p.err) atomicOr(p.err, FA_WS_WAIT_EXPIRED);
}

template <int D, int KIND, bool QBF16>
cudaError_t launch(const TreeParams& a, cudaStream_t st) {
  using C = TreeShape<D, KIND>;
  TreeTcParams kp;
  kp.a = a;
  kp.PT = kTtM / a.G;
  kp.alt = C::NG == 2 && a.T <= kp.PT;
  const long long slots = (long long)a.S * a.T;
  kp.q_box = (int)(slots < kp.PT ? slots : kp.PT);
  kp.tma_kv = a.R >= 64;
  CUtensorMap tq, tk, tv;
  memset(&tq, 0, sizeof(tq));
  memset(&tk, 0, sizeof(tk));
  memset(&tv, 0, sizeof(tv));
  // tensors [d2][d1][d0] of 16-bit values, or of bytes
  auto map = [&](CUtensorMap* m, const void* base, CUtensorMapDataType dt, int es, long long d0, long long d1,
                 long long d2, int b0, int b1, int b2) {
    const cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
    const cuuint64_t strides[2] = {(cuuint64_t)(d0 * es), (cuuint64_t)(d0 * d1 * es)};
    const cuuint32_t box[3] = {(cuuint32_t)b0, (cuuint32_t)b1, (cuuint32_t)b2};
    return tmap_encode_3d(m, dt, base, dims, strides, box, es == 1 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B);
  };
  const CUtensorMapDataType q_type = QBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  if (!map(&tq, a.q, q_type, 2, D, a.Hq, slots, 64, a.G, kp.q_box)) return cudaErrorInvalidValue;
  if (kp.tma_kv) {
    const CUtensorMapDataType type = C::QUANT ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : q_type;
    const int es = C::QUANT ? 1 : 2, d0 = C::ROW / es, b0 = C::QUANT ? C::ROW : 64;
    if (!map(&tk, a.k, type, es, d0, a.Hkv, a.R, b0, 1, 64) || !map(&tv, a.v, type, es, d0, a.Hkv, a.R, b0, 1, 64))
      return cudaErrorInvalidValue;
  }
  const cudaError_t e = once_per_device<21>([] {
    return cudaFuncSetAttribute(tree_tc_kernel<D, KIND, QBF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (e != cudaSuccess) return e;
  tree_tc_kernel<D, KIND, QBF16><<<a.ctas, C::NWARP * 32, C::SMEM, st>>>(kp, tq, tk, tv);
  return cudaGetLastError();
}

}  // namespace

bool tree_tc_shape(int D, int kind, int T, int G, int* rows, int* row_tiles, int* tile) {
  if (G > kTtM || !(D == 128 || (!tt_quant(kind) && (D == 64 || D == 256)))) return false;
  const int PT = kTtM / G, per = (D != 256 && T > PT ? 2 : 1) * PT;   // nodes of a row tile, of a unit
  *rows = per * G;
  *row_tiles = (T + per - 1) / per;
  *tile = 64;
  return true;
}

cudaError_t tree_tc_launch(const TreeParams& p, cudaStream_t st) {
  const bool b = p.q_bf16 != 0;
  if (p.kind == KV_BF16 || p.kind == KV_F16) {
    const bool bf16 = p.kind == KV_BF16;
    if (p.D == 64) return bf16 ? launch<64, KV_BF16, true>(p, st) : launch<64, KV_F16, false>(p, st);
    if (p.D == 128) return bf16 ? launch<128, KV_BF16, true>(p, st) : launch<128, KV_F16, false>(p, st);
    if (p.D == 256) return bf16 ? launch<256, KV_BF16, true>(p, st) : launch<256, KV_F16, false>(p, st);
  }
  if (p.kind == KV_I8) return b ? launch<128, KV_I8, true>(p, st) : launch<128, KV_I8, false>(p, st);
  if (p.kind == KV_I4) return b ? launch<128, KV_I4, true>(p, st) : launch<128, KV_I4, false>(p, st);
  if (p.kind == KV_F8) return b ? launch<128, KV_F8, true>(p, st) : launch<128, KV_F8, false>(p, st);
  return cudaErrorInvalidValue;
}

}  // namespace far
