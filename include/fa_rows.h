/*
 * fa_rows.h — row-indexed flash attention over a unified KV pool (C ABI).
 *
 * The operation ("llama.cpp 0.9.0 inference boundaries", section 1, the
 * ggml_flash_attn_ext_rows paragraph): every sequence's K/V rows share one
 * storage pool; each query slice carries its own integer kv_rows list naming
 * the pool rows it attends to; a negative row index is padding whose mask is
 * minus infinity.  The next paragraph of that section fixes that the result is
 * exact attention over the listed rows, not a lossy summary.
 *
 * Paged KV with 64-token pages and an INT8 cache: the v100llm article,
 * sections 1-2 ("FlashAttention 1.5 SM70 kernels", "Paged KV cache").
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers, row-major and contiguous, owned
 *    by the caller.  The library never allocates device memory, never
 *    synchronises, and enqueues all work on the given stream.
 *  - Argument errors are detected on the host before anything is launched and
 *    returned as a status; nothing is thrown across this boundary.  A failed
 *    launch returns FA_ERR_CUDA; fa_last_error() then names the CUDA error.
 *  - Row indices are NOT range-checked by the attention calls (that would cost
 *    a pass over the lists); fa_rows_validate() checks them on the device and
 *    reports through a status word, without trapping.
 *  - Every wait inside the tensor-core kernels is bounded in time (1 s by
 *    default, see fa_set_wait_limit_ns).  A wait that runs out is treated as a
 *    hang: the kernel leaves its pipeline, lets its own copies and MMAs drain,
 *    frees its tensor memory and sets FA_WS_WAIT_EXPIRED in the status word of
 *    the call's workspace (fa_rows_status reads it).  That call's outputs are
 *    then invalid; the call itself has already returned FA_OK, since the wait
 *    runs on the GPU after the launch.
 */
#ifndef FA_ROWS_H
#define FA_ROWS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* fa_stream_t; /* a cudaStream_t; NULL = legacy default stream */

typedef enum fa_status {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1,  /* null pointer, bad size, inconsistent shape        */
  FA_ERR_UNSUPPORTED = 2,  /* valid but outside the shapes/dtypes built here   */
  FA_ERR_WORKSPACE = 3,    /* workspace missing or smaller than required        */
  FA_ERR_INDEX_OOB = 4,    /* reported by fa_rows_validate through its status   */
  FA_ERR_CUDA = 5,         /* a CUDA launch or runtime call failed              */
  FA_ERR_WAIT_EXPIRED = 6  /* not returned by a launch: the code to report when
                            * a workspace status word holds FA_WS_WAIT_EXPIRED */
} fa_status;

/* Bits of the workspace status word (the first uint32 of every decode and
 * prefill workspace).  Sticky: set by any call on that workspace, cleared only
 * by fa_rows_workspace_init or fa_rows_status(..., clear = 1). */
#define FA_WS_WAIT_EXPIRED 1u  /* a bounded pipeline wait ran out; that call's outputs are invalid */

typedef enum fa_dtype { FA_F16 = 0, FA_BF16 = 1, FA_F32 = 2, FA_I8 = 3, FA_I4 = 4, FA_F8E4M3 = 5 } fa_dtype;

typedef enum fa_mask_kind {
  FA_MASK_NONE = 0,
  /* additive fp32 mask [S, Nq, L], aligned with list POSITION j (not pool row);
   * minus infinity removes an entry.  Section 1's "corresponding mask". */
  FA_MASK_DENSE = 1,
  /* bottom-right causal: the slice's Nq queries are the last Nq positions of
   * its n_s list entries, so query i sees list positions j <= n_s - Nq + i. */
  FA_MASK_CAUSAL = 2
} fa_mask_kind;

/*
 * Arguments of one row-indexed attention call.
 *
 *   q        [S, Nq, Hq, D]     FA_F16 or FA_BF16
 *   k, v     [R, Hkv, D]        the unified pool: FA_F16/FA_BF16 (same as q),
 *                               FA_I8 (int8 codes, then k_scale/v_scale), or
 *            [R, Hkv, D/2]      FA_I4 (two 4-bit codes per byte, element 2t in
 *                               the low nibble of byte t; D = 128 only), or
 *            [R, Hkv, D]        FA_F8E4M3 (OCP E4M3 bytes; D = 128 only)
 *   k_scale, v_scale            quantised pools only: fp16 bit patterns laid out
 *                               [R/64, Hkv, 64], i.e. the scale of (row r,
 *                               head g) sits at ((r/64)*Hkv + g)*64 + r%64;
 *                               value = code * scale (R must be a multiple of 64)
 *   kv_rows  [S, L] int32       pool row of list entry j of slice s; negative =
 *                               padding.  Duplicates count once per occurrence.
 *   kv_len   [S] int32 or NULL  n_s: entries at positions >= kv_len[s] are
 *                               padding (NULL: n_s = L)
 *   mask     [S, Nq, L] fp32    FA_MASK_DENSE only
 *   out      [S, Nq, Hq, D]     FA_F32, FA_BF16 or FA_F16
 *   lse      [S, Nq, Hq] fp32   optional natural-log log-sum-exp of the logits
 *
 * Query head h reads KV head h / (Hq/Hkv).  Logit of entry j for query i:
 * scale * <q, K[row]> (+ mask[s,i,j]).  A query with no visible entry gets
 * out = 0 and lse = -inf.
 *
 * n_valid_hint: optional host-side count of listed entries summed over all
 * slices (0 = unknown); it only steers how the list is split across SMs.
 */
typedef struct fa_rows_args {
  const void* q;
  fa_dtype q_dtype;
  const void* k;
  const void* v;
  fa_dtype kv_dtype;
  const uint16_t* k_scale;
  const uint16_t* v_scale;
  int64_t n_pool_rows;
  const int32_t* kv_rows;
  int32_t list_len;
  const int32_t* kv_len;
  fa_mask_kind mask_kind;
  const float* mask;
  float scale;
  void* out;
  fa_dtype out_dtype;
  float* lse;
  int32_t S, Nq, Hq, Hkv, D;
  int64_t n_valid_hint;
} fa_rows_args;

/*
 * Bytes of scratch (a device buffer, 256-byte aligned) that fa_rows_decode /
 * fa_rows_prefill need for these arguments; at least 256.  Layout: bytes
 * [0, 256) are the status block, whose first uint32 is the status word
 * (FA_WS_WAIT_EXPIRED; the next words are the calls' own scratch); when decode
 * splits the lists over several CTAs, one arrival counter per (slice, KV head)
 * follows, and from byte 16384 on the per-split partial results (behind the
 * counters where these need more).  The buffer must be ZERO-FILLED once after
 * allocation (fa_rows_workspace_init); every call leaves the counters at zero
 * again, an aborted one included, so calls of any arguments may use one
 * workspace that is large enough for each in turn.  One workspace must not be
 * used by two calls that can run at the same time.  Returns 0 and sets
 * fa_last_error() on invalid arguments.
 */
size_t fa_rows_workspace_size(const fa_rows_args* a, int is_prefill);
fa_status fa_rows_workspace_init(void* ws, size_t ws_bytes, fa_stream_t stream);

/*
 * Kernel launches one fa_rows_decode call with these arguments makes: 1, or 2
 * when the plan merges the list's splits in a kernel of its own (a
 * latency-bound 16-bit decode: one wave of CTAs, each over at most four
 * tiles), 0 when there is nothing to do; -1 (and fa_last_error()) on invalid
 * arguments.  Host-only: no device work, no stream.
 */
int fa_rows_decode_launches(const fa_rows_args* a);

/*
 * Enqueues on `stream` a copy of the workspace's status word into *d_status
 * (a device uint32) and, if `clear` is non-zero, then zeroes the word.  The
 * caller reads d_status once the stream has reached this point; a non-zero
 * FA_WS_WAIT_EXPIRED bit means a call on this workspace since the word was
 * last cleared had a pipeline wait run out, so its outputs are invalid.
 * ws_bytes must be at least 256.  No counterpart on the pages: the pages
 * describe no failure path.
 */
fa_status fa_rows_status(void* ws, size_t ws_bytes, uint32_t* d_status, int clear, fa_stream_t stream);

/*
 * Diagnostic: the time limit, in nanoseconds, of every bounded pipeline wait
 * in kernels launched after this call by any thread of the process (0 restores
 * the default of 1 s).  Lowering it to a few nanoseconds makes waits run out
 * on purpose, which exercises the abort path and the status word in tests.
 * The drain waits of an aborting kernel keep the 1 s default.
 * No counterpart on the pages.
 */
fa_status fa_set_wait_limit_ns(uint64_t limit_ns);

/*
 * Decode: few query rows per slice (Nq * Hq/Hkv <= 32).  Split-KV over the
 * list, online softmax per split, cross-split merge inside the same launch
 * (by the last split of each (slice, KV head) to finish), or, for a
 * latency-bound 16-bit decode, in a second kernel enqueued right after it on
 * the same stream (fa_rows_decode_launches tells which).
 * D in {64, 128, 256}; Hq/Hkv a power of two up to 32 (times Nq).
 */
fa_status fa_rows_decode(const fa_rows_args* a, void* ws, size_t ws_bytes, fa_stream_t stream);

/*
 * Decode for callers that cannot allocate device memory.  The pages have no
 * counterpart to this call; it exists for hosts that may not call cudaMalloc
 * (or any allocating routine) where they run attention: code inside a custom
 * device allocator or its callbacks, plugins whose framework owns every device
 * allocation, and latency-critical paths that cannot afford an allocation or
 * its failure.  Same arguments and results as fa_rows_decode, but the
 * split-merge scratch comes from a static device array (16 MiB and the counters) inside this
 * library (held on every GPU that loads it, until the process exits).
 * Arguments whose scratch would exceed 16 MiB are rejected with
 * FA_ERR_WORKSPACE before anything is launched.  The first call on a device
 * looks up the array's device address (cudaGetSymbolAddress), so make that
 * first call before any stream capture.  Each call zero-fills the part of the
 * array it uses; all calls share the array, so calls that overlap on the GPU
 * (other streams or threads) race and must be serialised by the caller.
 */
fa_status fa_rows_decode_static(const fa_rows_args* a, fa_stream_t stream);

/*
 * Prefill: many query rows per slice.  QK^T and PV on the tensor cores
 * (tcgen05, accumulators in tensor memory), K/V tiles gathered by row index.
 * D = 128, FA_BF16 or FA_F16 for q and the pool; Nq >= 1.  The workspace
 * (fa_rows_workspace_size(a, 1) = 256 bytes, zero-filled once) is required:
 * it holds the status word; a NULL ws is rejected with FA_ERR_WORKSPACE.
 * bf16 pools: the call first scans the listed V rows (one extra kernel, one
 * read of them) and writes words 1-3 of the status block as its own scratch:
 * when no listed V value is beyond f16's range (finite, 65536 or more) and
 * at most a quarter of the 128-entry KV tiles are gathered rather than one
 * contiguous pool run, V tiles are converted to f16 in shared memory and P
 * enters the PV product as one f16 value (11 significant bits; a bf16 V value
 * below 2^-14 in magnitude becomes an f16 subnormal, within 2^-25 of it);
 * otherwise V stays bf16 and P is the pair rn(P) + rn(P - rn(P)).
 */
fa_status fa_rows_prefill(const fa_rows_args* a, void* ws, size_t ws_bytes, fa_stream_t stream);

/*
 * Decode and prefill over one list per (slice, KV head): kv_rows [S, Hkv, L]
 * and kv_len [S, Hkv] (or NULL), so the heads of a slice may read different
 * rows (the lists that fa_kv_block_rows makes).  Everything else is as in
 * fa_rows_decode / fa_rows_prefill, the workspace and its size included, with
 * FA_MASK_NONE or FA_MASK_CAUSAL: a causal query i of KV head g sees positions
 * j <= kv_len[s, g] - Nq + i of its head's list, so each list must end with the
 * slice's Nq newest positions.  n_valid_hint counts the entries of all lists
 * divided by Hkv.  fa_rows_validate takes these lists with S * Hkv slices.
 * Prefill, bf16 pools: a KV tile of two contiguous 64-row runs (blocks) counts
 * as contiguous where fa_rows_prefill chooses between f16 and bf16 V, so lists
 * of whole blocks take f16 V and one f16 P.
 * Sparse attention over selected blocks (the v100llm article, section 5, and
 * the llama.cpp-v100 README's QSA attend to a selected subset of the context).
 */
fa_status fa_rows_decode_heads(const fa_rows_args* a, void* ws, size_t ws_bytes, fa_stream_t stream);
fa_status fa_rows_prefill_heads(const fa_rows_args* a, void* ws, size_t ws_bytes, fa_stream_t stream);

/*
 * Attention of the nodes of a drafted token tree, all in one pass over the list
 * (speculative decoding: the target model scores every node at once).  The
 * arguments are those of fa_rows_decode with Nq = T node slots a slice and
 * FA_MASK_NONE.  Of the slice's n_s entries the last m_s = n_nodes[s]
 * (n_nodes NULL: T; clamped to 0 .. T) are its nodes 0 .. m_s - 1 in order;
 * their K/V rows have been appended.  Node t sees the entries before these, and
 * of the nodes itself, parent[s,t], that one's parent and so on:
 *   j < n_s - m_s,  or  j = n_s - m_s + u  with u = t or an ancestor of t.
 * A parent outside 0 .. t-1 makes t a root.  Padding entries are not seen, a
 * node's own one included; n_s < m_s leaves the first m_s - n_s nodes without
 * entries.  Slots t >= m_s, and nodes that see nothing, get out = 0 and
 * lse = -inf.
 *   parent   [S, T] int32, n_nodes [S] int32 or NULL; T up to 256
 *   pools    every kind of fa_rows_args, D <= 256 with 16-byte multiples per
 *            (row, KV head); S * Hkv * T * Hq / Hkv * L / 1024 must fit int32.
 *            Tensor cores: D 64, 128 and 256 of 16-bit pools and D 128 of
 *            quantised ones, with Hq / Hkv up to 128 and q 16-byte aligned.  Every
 *            other call runs on the CUDA cores, tens of times slower: INT8, INT4
 *            and E4M3 at D 64 and 256, other D, larger groups, unaligned q
 *   ws       fa_rows_tree_workspace_size bytes, 256-byte aligned, zero-filled
 *            once; one workspace may serve this call and fa_rows_decode in turn
 * The lists are cut into equal shares for all SMs whatever their lengths; two
 * launches.  Equal calls give equal bits.  On the tensor cores a weight is a pair
 * of 16-bit values over 16-bit pools, and over quantised ones, times its V scale,
 * one f16 value (off by up to 2^-12).  Values that are not finite reach the
 * nodes that see them alone: an infinite V gives an infinity, a NaN, or
 * infinities of both signs, a NaN.
 */
size_t fa_rows_tree_workspace_size(const fa_rows_args* a);
fa_status fa_rows_tree(const fa_rows_args* a, const int32_t* parent, const int32_t* n_nodes, void* ws, size_t ws_bytes,
                       fa_stream_t stream);

/*
 * The path of each drafted tree that the target model agrees with, greedily:
 * node 0 (the token of the last step) is on it; a node c on it is followed by
 * its child t (parent[t] = c < t) with token[t] = target[c], where several are
 * by the one with the smallest number, and the path ends where there is none.
 *   parent, token, target  [S, T] int32; target[s,t]: the target model's token
 *                          after node t (from the logits of fa_rows_tree's pass)
 *   n_nodes  [S] int32 or NULL (T nodes); T up to 256
 *   kv_len   [S] int32 or NULL: list lengths with the nodes appended
 *   path     [S, T] the path's nodes, then -1;  n_path [S] how many
 *   next     [S] target of the last node of the path (no nodes: -1)
 *   len_out  [S] kv_len - m_s + n_path, at least 0; NULL exactly when kv_len is
 */
fa_status fa_tree_accept(const int32_t* parent, const int32_t* token, const int32_t* target, const int32_t* n_nodes,
                         int32_t S, int32_t T, const int32_t* kv_len, int32_t* path, int32_t* n_path, int32_t* next,
                         int32_t* len_out, fa_stream_t stream);

/*
 * Arrays that copies inside the pool work on.  FA_KV_ROWS: [R, row_bytes], a
 * pool's K or V (row_bytes = bytes of one row, all heads, a multiple of 16).
 * FA_KV_SCALES: the fp16 [R/64, Hkv, 64] of a quantised pool (row_bytes = 2 *
 * Hkv).  FA_KV_PAGES: one item for each 64-row page (row_bytes = bytes of an
 * item, a multiple of 16): block bounds.  Base pointers are 16-byte aligned.
 */
typedef enum fa_kv_layout { FA_KV_ROWS = 0, FA_KV_SCALES = 1, FA_KV_PAGES = 2 } fa_kv_layout;
typedef struct fa_kv_array {
  void* data;
  int64_t row_bytes;
  int32_t layout;
} fa_kv_array;

/*
 * Moves the rows of the accepted nodes to the first entries of the list's tail,
 * in place: for i < n_path[s] the row of entry n_s - m_s + i gets what the row
 * of entry n_s - m_s + path[s,i] held before the call (all of a slice's rows
 * are read before one is written).  The cache is then that of n_s - m_s +
 * n_path[s] tokens (fa_tree_accept's len_out) with unchanged lists.  Nodes
 * outside 0 .. m_s-1, entries outside the list and rows outside the pool are
 * skipped.  The tails of two slices must not share rows, nor two arrays memory.
 *   arrays   all layers' FA_KV_ROWS and FA_KV_SCALES arrays
 *   kv_rows  [S, list_len]; kv_len [S] or NULL (list_len) with the nodes
 *   n_nodes, path, n_path, T as in fa_tree_accept
 */
fa_status fa_kv_tree_keep(const fa_kv_array* arrays, int32_t n_arrays, int64_t n_pool_rows, const int32_t* kv_rows,
                          int32_t S, int32_t list_len, const int32_t* kv_len, const int32_t* n_nodes, int32_t T,
                          const int32_t* path, const int32_t* n_path, fa_stream_t stream);

/*
 * Page tables whose sequences share pages.  A page state of P pages is int32
 * [4 + 2 P]: word 0 the pages in the stack of free ones, word 1 the requests so
 * far that found no page, two zeros; P reference counts (page-table entries that
 * name the page); the stack, its top last (-1 past it).  P up to 2^25, max_pages
 * below that, and a table's entries fit int32.  A
 * sequence of n tokens holds the first ceil(n / 64) entries of its table row
 * (seq_len is clamped to 0 .. 64 * max_pages).  Page ids outside 0 .. P-1 are
 * entries without a page.  Each call reads tables, lengths and a state and
 * writes the next ones elsewhere: outputs overlap neither each other nor the
 * inputs.  A partly filled last page is to have one holder; fa_kv_fork sees to
 * that.
 *
 * fa_kv_pages_init: all pages free, page 0 on top.
 *
 * fa_kv_fork: sequence i of the n_new next ones continues old sequence src[i]
 * (outside 0 .. n_seq-1: is empty); the old ones are given up.  Whole pages are
 * shared.  A partly filled last page stays with the first i that continues its
 * sequence, if that was its only holder; every other i takes a page from the
 * stack, in the order of i, and copies names what to copy into it.  One that
 * finds none keeps its whole pages only (its length is cut to them), and word 1
 * counts it.  Pages without holders are then pushed, in increasing order.
 *   src       [n_new] int32
 *   table_out [n_new, max_pages], -1 past a sequence's pages; len_out [n_new]
 *   copies    [3, n_new]: source page, destination page and rows for
 *             fa_kv_copy_pages, before anything else is written to the pool (a
 *             source may be free by now); -1, -1, 0 where i copies nothing
 *
 * fa_kv_free: sequences with done[i] != 0 give up their pages, which are pushed
 * in increasing order where no holder is left; their rows become -1, their
 * lengths 0.
 *
 * fa_kv_cut: sequence i keeps its first keep[i] tokens (clamped to 0 .. its
 * length) and gives up the pages past them, as fa_kv_free does: what fa_kv_tree_keep
 * is followed by, with fa_tree_accept's lengths.  Entries past the pages it keeps
 * become -1.  Where the cut goes through a page that others hold too, fork before
 * growing: each then gets a last page of its own.
 *
 * fa_kv_grow: sequence i gets add[i] (clamped to 0 .. max_add) more tokens and
 * pages from the stack for them, in the order of i.  Where fewer are left than
 * it and those before it ask for, it does not grow and word 1 counts its pages;
 * nor does one that would pass max_pages (not counted).
 *   rows      [n_seq, max_add]: pool rows of the new tokens (fa_kv_append's
 *             dst_rows), -1 past add[i], where i did not grow and where an entry
 *             has no page
 *
 * fa_kv_compact: pages with a count above 0 move to ids 0 .. live-1: the k-th
 * free id below live takes the k-th live page at or past it.  The tables given
 * are rewritten; remap serves others.
 *   moves     [3, P / 2]: pages from and to, and 64 rows, for
 *             fa_kv_copy_pages (sources and destinations are apart); -1, -1, 0
 *             past them
 *   remap     [P]: a page's new id, -1 for a free one
 */
fa_status fa_kv_pages_init(int32_t* pages, int32_t n_pages, fa_stream_t stream);
fa_status fa_kv_fork(const int32_t* page_table, const int32_t* seq_len, int32_t n_seq, int32_t max_pages,
                     const int32_t* src, int32_t n_new, const int32_t* pages, int32_t n_pages, int32_t* table_out,
                     int32_t* len_out, int32_t* pages_out, int32_t* copies, fa_stream_t stream);
fa_status fa_kv_free(const int32_t* page_table, const int32_t* seq_len, int32_t n_seq, int32_t max_pages,
                     const int32_t* done, const int32_t* pages, int32_t n_pages, int32_t* table_out, int32_t* len_out,
                     int32_t* pages_out, fa_stream_t stream);
fa_status fa_kv_cut(const int32_t* page_table, const int32_t* seq_len, int32_t n_seq, int32_t max_pages,
                    const int32_t* keep, const int32_t* pages, int32_t n_pages, int32_t* table_out, int32_t* len_out,
                    int32_t* pages_out, fa_stream_t stream);
fa_status fa_kv_grow(const int32_t* page_table, const int32_t* seq_len, int32_t n_seq, int32_t max_pages,
                     const int32_t* add, int32_t max_add, const int32_t* pages, int32_t n_pages, int32_t* table_out,
                     int32_t* len_out, int32_t* pages_out, int32_t* rows, fa_stream_t stream);
fa_status fa_kv_compact(const int32_t* page_table, const int32_t* seq_len, int32_t n_seq, int32_t max_pages,
                        const int32_t* pages, int32_t n_pages, int32_t* table_out, int32_t* pages_out, int32_t* moves,
                        int32_t* remap, fa_stream_t stream);

/*
 * Copies pages inside the pool, for every array given (all layers' K and V,
 * scales, bounds): page copies[1,i] gets page copies[0,i], its first
 * copies[2,i] rows (FA_KV_SCALES and FA_KV_PAGES arrays: all of it).  Pairs with
 * a page outside 0 .. n_pool_pages-1, of a page with itself or with no rows are
 * skipped.  No page may be the destination of two pairs, or of one and the
 * source of another.
 *   copies   [3, n_copies] int32 (fa_kv_fork's copies, fa_kv_compact's moves)
 */
fa_status fa_kv_copy_pages(const fa_kv_array* arrays, int32_t n_arrays, int64_t n_pool_pages, const int32_t* copies,
                           int32_t n_copies, fa_stream_t stream);

/*
 * Attention weight received by each list entry, accumulated:
 *   acc[s, g, j] = decay * acc[s, g, j] + sum over i and the heads h of group g
 *                  of exp(scale * <q[s,i,h], K[row_j, g]> + mask - lse[s,i,h])
 * for every list position j < n_s, where lse [S, Nq, Hq] is what fa_rows_decode
 * or fa_rows_prefill wrote for the same arguments: each term is the softmax
 * weight that call gave the entry.  Of a, the fields v, v_scale, out, out_dtype
 * and lse are not read.  Terms that the mask, the causal limit or a padding
 * entry removes are zero, and so are those of a query whose lse is minus
 * infinity; positions at or past n_s keep their acc.  decay = 1 accumulates;
 * decay = 0 overwrites (acc is not read).  With S * Nq = 0 nothing is done.
 * One list per slice (kv_rows [S, L]): lists per KV head have no such call.
 * A term is as exact as lse, whose rounding (|lse| * 2^-24) is an error of the
 * term's exponent: a dense mask that adds a number of large magnitude to every
 * entry a query sees (-1e9 for a padded query, say) leaves no room in lse for
 * the rest, so hide entries with minus infinity.
 *   acc      [S, Hkv, L] fp32
 *   pools    every kind of fa_rows_args, D <= 256 with 16-byte multiples per
 *            (row, KV head); any mask kind; any Nq and Hq / Hkv; L and Nq * Hq
 *            up to 2^30.  D 64, 128 and 256 without a dense mask, with 16-byte
 *            aligned q and at most 128 (D 256: 64) query heads per KV head,
 *            take the tensor cores
 *   ws       256 bytes, zero-filled once (it holds the status word)
 * The order of the sums is fixed: equal calls give equal bits.
 */
fa_status fa_rows_weights(const fa_rows_args* a, const float* lse, float decay, float* acc, void* ws, size_t ws_bytes,
                          fa_stream_t stream);

/*
 * Range check of the lists (section 1: negative = padding; anything else must
 * name a pool row).  d_status is a device int64[2] that this call overwrites:
 * [0] = number of entries with kv_rows >= n_pool_rows (within kv_len),
 * [1] = flat index s*L + j of the first such entry, or -1.
 * Returns FA_OK once the check is enqueued; the caller reads d_status.
 */
fa_status fa_rows_validate(const fa_rows_args* a, int64_t* d_status, fa_stream_t stream);

/*
 * Page tables -> row lists (v100llm article, section 2: 64-token pages).
 * page_table [n_seq, max_pages] int32 page ids; seq_len [n_seq] int32 (device).
 * kv_rows [n_seq, list_len] is written as page_id*page_size + j%page_size for
 * j < seq_len[s] and -1 elsewhere.  seq_len values above max_pages*page_size
 * are clamped to it.
 */
fa_status fa_kv_page_table_to_rows(const int32_t* page_table, int32_t max_pages, const int32_t* seq_len,
                                   int32_t n_seq, int32_t page_size, int32_t* kv_rows, int32_t list_len,
                                   fa_stream_t stream);

/*
 * INT8 KV quantisation, per (row, KV head) with an fp16 scale (value = q*s):
 * s = fp16_rne(min(amax/127, 65504)) with amax/127 one fp32 division;
 * q = clamp(rint_half_even(x/s), -127, 127) with x/s one fp32 division;
 * s = 0 gives q = 0.
 *   x        [n_rows, Hkv, D] FA_F16 or FA_BF16 (x_dtype)
 *   dst_rows [n_rows] int32 pool rows to write, negative or >= R = skip;
 *            NULL = row i
 *   q        [R, Hkv, D] int8 pool; scale the fp16 layout of fa_rows_args.
 * This is also the KV append of a ubatch into an INT8 pool.
 */
fa_status fa_kv_quantize_int8(const void* x, fa_dtype x_dtype, int64_t n_rows, int32_t Hkv, int32_t D,
                              const int32_t* dst_rows, int8_t* q, uint16_t* scale, int64_t n_pool_rows,
                              fa_stream_t stream);

/* out[r, g, d] = float(q[r, g, d]) * float(scale of (r, g)), exact in fp32. */
fa_status fa_kv_dequantize_int8(const int8_t* q, const uint16_t* scale, int64_t n_rows, int32_t Hkv, int32_t D,
                                float* out, fa_stream_t stream);

/*
 * INT4 KV quantisation for the paged INT4 pool the v100llm article names
 * (section 2, "INT4/INT8 paged path"; it gives no rule): the INT8 rule above
 * with 7 in place of 127 (s = fp16_rne(min(amax/7, 65504)), codes in -7..7),
 * stored as two's-complement nibbles, element 2t in the low nibble of byte t.
 *   q        [R, Hkv, D/2] uint8 pool; scale the fp16 layout of fa_rows_args.
 * D must be even and <= 256; negative dst_rows entries are skipped.
 */
fa_status fa_kv_quantize_int4(const void* x, fa_dtype x_dtype, int64_t n_rows, int32_t Hkv, int32_t D,
                              const int32_t* dst_rows, uint8_t* q, uint16_t* scale, int64_t n_pool_rows,
                              fa_stream_t stream);

/* out[r, g, d] = float(nibble code) * float(scale of (r, g)), exact in fp32. */
fa_status fa_kv_dequantize_int4(const uint8_t* q, const uint16_t* scale, int64_t n_rows, int32_t Hkv, int32_t D,
                                float* out, fa_stream_t stream);

/*
 * FP8 E4M3 KV quantisation.  "llama.cpp 0.9.0 inference boundaries"
 * (section 4) adds the OCP FP8 E4M3 type in saturating mode and leaves its KV
 * use and scaling to later work; the rule here mirrors the INT8 one:
 * s = fp16_rne(min(amax/448, 65504)); code = E4M3 of x/s (one fp32 division,
 * round to nearest even, saturating to +-448, NaN -> 0x7f); s = 0 gives 0.
 *   q        [R, Hkv, D] E4M3 bytes; scale the fp16 layout of fa_rows_args.
 */
fa_status fa_kv_quantize_fp8(const void* x, fa_dtype x_dtype, int64_t n_rows, int32_t Hkv, int32_t D,
                             const int32_t* dst_rows, uint8_t* q, uint16_t* scale, int64_t n_pool_rows,
                             fa_stream_t stream);

/* out[r, g, d] = float(E4M3 value of q[r, g, d]) * float(scale of (r, g)), exact in fp32. */
fa_status fa_kv_dequantize_fp8(const uint8_t* q, const uint16_t* scale, int64_t n_rows, int32_t Hkv, int32_t D,
                               float* out, fa_stream_t stream);

/*
 * Sparse row-list builder (v100llm article, section 5: anchor + recent + sink
 * selection; the llama.cpp-v100 README's QSA reads such a subset of a long
 * context).  For each slice s with n = min(n_len[s], n_max) positions
 * (n_len NULL: n = n_max): positions 0 .. sinks-1, the k positions of
 * [sinks, n - recent) with the largest score[s, pos], and n-recent .. n-1,
 * in increasing position order, padded with -1.  Ties in score go to the
 * smaller position; a NaN score ranks below every number.  Slices with no
 * more than k middle positions list every position.
 *   score    [S, n_max] fp32, caller-provided (the learned indexer that would
 *            produce it is not part of this library)
 *   row_map  [S, n_max] int32 position -> pool row, or NULL (row = position)
 *   kv_rows  [S, list_len] int32 output; list_len >= sinks + recent + k
 *   ws       scratch of fa_kv_sparse_rows_workspace_size(S, n_max) bytes
 *            (16-byte aligned; its contents need no initialisation): each
 *            slice is then spread over blocks of 8192 positions (several
 *            launches on the stream).  NULL: one CTA per slice, no scratch.
 * The output is bit-exact (an integer selection) either way.
 */
size_t fa_kv_sparse_rows_workspace_size(int32_t S, int32_t n_max);
fa_status fa_kv_sparse_rows(const float* score, int32_t n_max, const int32_t* n_len, int32_t S, int32_t sinks,
                            int32_t recent, int32_t k, const int32_t* row_map, int32_t* kv_rows, int32_t list_len,
                            void* ws, size_t ws_bytes, fa_stream_t stream);

/*
 * Eviction from row lists by accumulated weight.  Of each slice's
 * n = min(kv_len[s], list_len) entries (kv_len NULL: list_len), these are kept:
 * list positions 0 .. sinks-1, positions n-recent .. n-1, and of the positions
 * between them the k with the largest total, the sum of acc over the KV heads
 * rounded once to fp32 (formed with at least 48 bits).  Ties go to the smaller
 * position; a NaN total ranks below every number; padding entries (negative
 * rows) are never kept.  A slice with no more entries than that keeps them all.
 *   acc       [S, Hkv, list_len] fp32 (fa_rows_weights), kv_rows [S, list_len]
 *   rows_out  [S, out_len] the kept entries' rows in list order, then -1
 *   len_out   [S] how many were kept
 *   acc_out   [S, Hkv, out_len] their acc, then 0: the accumulator that goes
 *             with rows_out
 *   kept      [S, out_len] their list positions, then -1; or NULL
 *   freed     [S, list_len] the other entries' rows in list order, then -1; or
 *             NULL.  These pool rows may be reused.
 * out_len >= sinks + recent + k.  Outputs must overlap neither each other nor
 * the inputs.  No workspace.
 */
fa_status fa_kv_evict(const float* acc, const int32_t* kv_rows, const int32_t* kv_len, int32_t S, int32_t Hkv,
                      int32_t list_len, int32_t sinks, int32_t recent, int32_t k, float* acc_out, int32_t* rows_out,
                      int32_t* len_out, int32_t out_len, int32_t* kept, int32_t* freed, fa_stream_t stream);

/*
 * Elementwise bounds of the keys of 64-row pages (the blocks of
 * fa_kv_block_scores): for each listed page, kmin and kmax[page, g, d] over the
 * page's first fill[i] rows (fill NULL: 64; clamped to 0 .. 64).  Exact for a
 * 16-bit pool; for a quantised pool the bounds of code * scale rounded outward
 * (down for kmin, up for kmax) to bound_dtype.  A NaN key makes its bounds
 * NaN.  Pages with fill <= 0, and page ids below 0 or at or past
 * n_pool_rows / 64, are skipped: their bounds are left as they were.  A page
 * listed twice must have the same fill both times.
 *   k, k_scale  the K pool as in fa_rows_args; n_pool_rows a multiple of 64
 *   pages, fill [n_pages] int32
 *   kmin, kmax  [n_pool_rows / 64, Hkv, D] FA_F16 or FA_BF16 (the pool's dtype
 *               for a 16-bit pool)
 * Called for the touched pages after an append.
 */
fa_status fa_kv_block_bounds(const void* k, fa_dtype kv_dtype, const uint16_t* k_scale, int64_t n_pool_rows,
                             int32_t Hkv, int32_t D, const int32_t* pages, const int32_t* fill, int32_t n_pages,
                             void* kmin, void* kmax, fa_dtype bound_dtype, fa_stream_t stream);

/*
 * Scores of a sequence's blocks for each query slice and KV head:
 *   score[s, g, b] = max over the slice's queries i and the heads h of group g of
 *                    sum_d max(q_d, 0) * kmax[page, g, d] + min(q_d, 0) * kmin[page, g, d],
 * which no dot product of one of those queries with a key of the block exceeds
 * (but for fp32 rounding).  A component takes the bound of its sign and a zero
 * takes none, so an infinite bound (fa_kv_block_bounds rounds a key beyond the
 * bounds' dtype to one) makes the score plus infinity or leaves it a number.
 * Minus infinity for b >= ceil(seq_len[s] / 64) and for page ids below 0 or at
 * or past n_pool_pages; NaN where q or a bound of the block is NaN, or where
 * infinite terms of both signs meet.
 *   q          [S, Nq, Hq, D] and the bounds in the same dtype, D in {64,128,256}
 *   page_table [n_seq, max_pages] int32; slice s reads row slice_seq[s], or row s
 *              when slice_seq is NULL (several slices of one sequence: prompt tiles).
 *              A slice whose slice_seq is outside 0 .. n_seq-1 scores minus infinity.
 *   seq_len    [S] int32: positions that slice s may see
 *   score      [S, Hkv, max_pages] fp32; with S * Nq = 0 nothing is written
 *   ws         256 bytes, zero-filled once (it holds the status word)
 */
fa_status fa_kv_block_scores(const void* q, fa_dtype q_dtype, int32_t S, int32_t Nq, int32_t Hq, int32_t Hkv, int32_t D,
                             const void* kmin, const void* kmax, int64_t n_pool_pages, const int32_t* page_table,
                             int32_t n_seq, int32_t max_pages, const int32_t* seq_len, const int32_t* slice_seq,
                             float* score, void* ws, size_t ws_bytes, fa_stream_t stream);

/*
 * Row lists of the best blocks of each (slice, KV head).  Of the
 * nb = ceil(min(seq_len[s], 64 * max_pages) / 64) blocks: the first
 * sink_blocks, the last recent_blocks, and of those between them the k with
 * the largest score (ties to the smaller block; NaN below every number); all
 * when there are no more.  Their rows page * 64 + t are listed in position
 * order, the sequence's last block up to seq_len.
 *   score    [S, Hkv, max_pages] fp32 (fa_kv_block_scores)
 *   kv_rows  [S, Hkv, list_len] int32, padded with -1; a block whose page id is
 *            negative (or page * 64 + 63 past int32) is listed as -1 entries
 *   kv_len   [S, Hkv] int32: entries listed
 * list_len >= 64 * (sink_blocks + recent_blocks + k).  page_table, seq_len and
 * slice_seq as in fa_kv_block_scores.  The lists feed fa_rows_decode_heads and
 * fa_rows_prefill_heads (causal: with recent_blocks >= 1 + ceil(Nq / 64) every
 * list ends with the slice's Nq newest positions).
 */
fa_status fa_kv_block_rows(const float* score, const int32_t* page_table, int32_t n_seq, int32_t max_pages,
                           const int32_t* seq_len, const int32_t* slice_seq, int32_t S, int32_t Hkv,
                           int32_t sink_blocks, int32_t recent_blocks, int32_t k, int32_t* kv_rows, int32_t* kv_len,
                           int32_t list_len, fa_stream_t stream);

/*
 * KV append for 16-bit pools: pool[dst_rows[i]] = x[i] for i < n_rows
 * (negative dst = skip).  x and pool are [*, Hkv, D] of the same 16-bit dtype.
 */
fa_status fa_kv_append(const void* x, fa_dtype dtype, int64_t n_rows, int32_t Hkv, int32_t D,
                       const int32_t* dst_rows, void* pool, int64_t n_pool_rows, fa_stream_t stream);

const char* fa_status_string(fa_status s);
/* Text of the last error seen by the calling thread ("" if none). */
const char* fa_last_error(void);
/* Library build tag, e.g. "fa_rows sm_103a". */
const char* fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_ROWS_H */
