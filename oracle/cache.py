"""Cache reduction in fp64: attention weight per list entry, eviction by it, key
bounds and scores of 64-row blocks, block row lists, attention over one list
per KV head.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Written from the definitions: the softmax weight of an entry is
exp(logit - LSE) with the logits of ``attend_rows``; a block's score is the
largest value that q . x can take for x between the block's elementwise key
bounds.  Selection rules are those of ``select_rows`` (ties to the smaller
position, NaN below every number).
"""
from __future__ import annotations

from typing import Optional

import numpy as np

from .attention import attend_rows, visible_positions
from .kvcache import PAGE, widen


def attend_rows_heads(q, k, v, kv_rows, scale, *, causal=False, kv_len=None, query_rows=None, n_query=None,
                      kv_format=None):
    """``attend_rows`` with one list per (slice, KV head): kv_rows [S, Hkv, L], kv_len [S, Hkv] or None."""
    Hkv = k.shape[1]
    G = q.shape[2] // Hkv
    parts = [attend_rows(q[:, :, g * G:(g + 1) * G], k[:, g:g + 1], v[:, g:g + 1], kv_rows[:, g], scale,
                         causal=causal, kv_len=None if kv_len is None else kv_len[:, g], query_rows=query_rows,
                         n_query=n_query, kv_format=kv_format) for g in range(Hkv)]
    return np.concatenate([p[0] for p in parts], axis=2), np.concatenate([p[1] for p in parts], axis=2)


def attention_weights(q, k, kv_rows, scale, lse, *, mask=None, causal=False, kv_len=None, n_pool_rows=None):
    """w [S, Hkv, L]: the weight every list position received, summed over the
    slice's queries and the heads of each group (0 at positions past kv_len)."""
    S, Nq, Hq, D = q.shape
    R, Hkv, _ = k.shape
    G = Hq // Hkv
    L = kv_rows.shape[1]
    w = np.zeros((S, Hkv, L))
    for s in range(S):
        n_s = L if kv_len is None else int(min(max(int(kv_len[s]), 0), L))
        rows = kv_rows[s, :n_s].astype(np.int64)
        pos = np.arange(n_s)[(rows >= 0) & (rows < R)]
        rows = rows[pos]
        for h in range(Hq):
            for i in range(Nq):
                see = np.full(len(pos), lse[s, i, h] > -np.inf)
                if causal:
                    see &= pos < visible_positions(n_s, Nq, i, True)
                x = scale * (k[rows, h // G] @ q[s, i, h])
                if mask is not None:
                    see &= mask[s, i, pos] > -np.inf
                    x = x + mask[s, i, pos].astype(np.float64)
                w[s, h // G, pos[see]] += np.exp(x[see] - float(lse[s, i, h]))
    return w


def _best(values, candidates, k):
    """The k candidates with the largest values, in increasing order."""
    def rank(c):
        x = float(values[c])
        return (1, 0.0, c) if x != x else (0, -x, c)
    return sorted(sorted(candidates, key=rank)[:k])


def evict(acc, kv_rows, kv_len, sinks, recent, k, out_len):
    """(rows [S, out_len], len [S], acc [S, Hkv, out_len], kept [S, out_len], freed [S, L])."""
    S, Hkv, L = acc.shape
    rows = np.full((S, out_len), -1, np.int32)
    kept = np.full((S, out_len), -1, np.int32)
    freed = np.full((S, L), -1, np.int32)
    length = np.zeros(S, np.int32)
    out = np.zeros((S, Hkv, out_len), acc.dtype)
    for s in range(S):
        n = L if kv_len is None else int(min(max(int(kv_len[s]), 0), L))
        live = [j for j in range(n) if kv_rows[s, j] >= 0]
        lo, hi = min(sinks, n), max(min(sinks, n), n - recent)
        with np.errstate(over="ignore", invalid="ignore"):
            total = acc[s].astype(np.float64).sum(axis=0).astype(np.float32)
        middle = _best(total, [j for j in live if lo <= j < hi], k)
        keep = [j for j in live if j < lo] + middle + [j for j in live if j >= hi]
        gone = sorted(set(live) - set(keep))
        length[s] = len(keep)
        rows[s, :len(keep)] = kv_rows[s, keep]
        kept[s, :len(keep)] = keep
        out[s, :, :len(keep)] = acc[s][:, keep]
        freed[s, :len(gone)] = kv_rows[s, gone]
    return rows, length, out, kept, freed


def round_outward(x: np.ndarray, up: bool, fmt: str) -> np.ndarray:
    """Bits of the nearest value of the 16-bit format that is >= x (up) or <= x, for finite x."""
    every = np.arange(1 << 16, dtype=np.uint16)
    val = widen(every, fmt)
    fine = ~np.isnan(val) & ~((val == 0) & (every != 0))
    order = np.argsort(val[fine], kind="stable")
    v, b = val[fine][order], every[fine][order]
    at = np.searchsorted(v, x, side="left") if up else np.searchsorted(v, x, side="right") - 1
    return b[at]


def block_bounds(k, pages, fill, kmin, kmax, fmt):
    """k float64 [R, Hkv, D] values; kmin, kmax uint16 bits [R/64, Hkv, D], updated copies returned."""
    kmin, kmax = kmin.copy(), kmax.copy()
    for i, page in enumerate(pages):
        m = PAGE if fill is None else min(max(int(fill[i]), 0), PAGE)
        if not 0 <= page < kmin.shape[0] or m == 0:
            continue
        x = k[page * PAGE:page * PAGE + m]
        kmin[page] = round_outward(x.min(axis=0), False, fmt)
        kmax[page] = round_outward(x.max(axis=0), True, fmt)
    return kmin, kmax


def block_scores(q, kmin, kmax, page_table, seq_len, slice_seq: Optional[np.ndarray] = None):
    """q, kmin, kmax float64; returns score [S, Hkv, max_pages].

    A component takes the bound of its sign, a zero none, whatever the other
    bound is; NaN where q or either bound is NaN, or infinite terms of both
    signs meet.
    """
    S, Nq, Hq, D = q.shape
    P, Hkv, _ = kmin.shape
    G = Hq // Hkv
    n_seq, NB = page_table.shape
    out = np.full((S, Hkv, NB), -np.inf)
    for s in range(S):
        t = s if slice_seq is None else int(slice_seq[s])
        if not 0 <= t < n_seq:
            continue
        for b in range(min(NB, -(-max(int(seq_len[s]), 0) // PAGE))):
            page = int(page_table[t, b])
            if not 0 <= page < P:
                continue
            for h in range(Hq):
                lo, hi = kmin[page, h // G], kmax[page, h // G]
                for i in range(Nq):
                    x = q[s, i, h]
                    with np.errstate(invalid="ignore"):
                        term = np.where(x > 0, x * hi, np.where(x < 0, x * lo, x))
                        best = float(term.sum())
                    if np.isnan(lo).any() or np.isnan(hi).any():
                        best = float("nan")
                    out[s, h // G, b] = best if best != best else max(out[s, h // G, b], best)
    return out


def block_rows(score, page_table, seq_len, sinks, recent, k, list_len, slice_seq: Optional[np.ndarray] = None):
    """(kv_rows int32 [S, Hkv, list_len], kv_len int32 [S, Hkv])."""
    S, Hkv, NB = score.shape
    rows = np.full((S, Hkv, list_len), -1, np.int32)
    length = np.zeros((S, Hkv), np.int32)
    for s in range(S):
        t = s if slice_seq is None else int(slice_seq[s])
        n = min(max(int(seq_len[s]), 0), NB * PAGE) if 0 <= t < page_table.shape[0] else 0
        nb = -(-n // PAGE)
        lo, hi = min(sinks, nb), max(min(sinks, nb), nb - recent)
        for g in range(Hkv):
            chosen = list(range(lo)) + _best(score[s, g], range(lo, hi), k) + list(range(hi, nb))
            at = 0
            for b in chosen:
                for o in range(min(PAGE, n - b * PAGE)):
                    page = int(page_table[t, b])
                    rows[s, g, at] = page * PAGE + o if 0 <= page <= (2 ** 31 - 64) // PAGE else -1
                    at += 1
            length[s, g] = at
    return rows, length
