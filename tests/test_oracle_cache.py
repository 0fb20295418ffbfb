"""Pins of the oracle's cache-reduction functions: closed forms, invariants and hand-worked cases (CPU)."""
import numpy as np
import pytest

import oracle
import synth


def _small(seed, **kw):
    p = synth.random_problem(seed, S=2, Nq=3, Hq=4, Hkv=2, D=8, R=40, L=13, **kw)
    return p, oracle.widen_bf16(p.q), oracle.widen_bf16(p.k), oracle.widen_bf16(p.v)


@pytest.mark.parametrize("kw", [dict(), dict(causal=True), dict(kv_len=True), dict(with_mask=True, neg_inf_frac=0.3)])
def test_weights_of_a_query_sum_to_one_and_give_the_output(kw):
    p, q, k, v = _small(3, **kw)
    out, lse = oracle.attend_rows(q, k, v, p.kv_rows, p.scale, mask=p.mask, causal=p.causal, kv_len=p.kv_len)
    w = oracle.attention_weights(q, k, p.kv_rows, p.scale, lse, mask=p.mask, causal=p.causal, kv_len=p.kv_len)
    rows_with = np.isfinite(lse).reshape(p.S, p.Nq, p.Hkv, -1).sum(axis=(1, 3))
    assert np.allclose(w.sum(axis=2), rows_with, rtol=1e-12, atol=1e-12)
    # the weighted values of a group are the sum of its outputs
    got = np.einsum("sgj,sjgd->sgd", w, np.where((p.kv_rows >= 0)[..., None, None], v[np.maximum(p.kv_rows, 0)], 0.0))
    want = out.reshape(p.S, p.Nq, p.Hkv, -1, p.D).sum(axis=(1, 3))
    assert np.allclose(got, want, rtol=1e-10, atol=1e-12)


def test_head_lists_equal_plain_lists_when_every_head_has_the_same():
    p, q, k, v = _small(4, causal=True, kv_len=True)
    rows = np.repeat(p.kv_rows[:, None], p.Hkv, axis=1)
    lens = np.repeat(p.kv_len[:, None], p.Hkv, axis=1)
    a = oracle.attend_rows_heads(q, k, v, rows, p.scale, causal=True, kv_len=lens)
    b = oracle.attend_rows(q, k, v, p.kv_rows, p.scale, causal=True, kv_len=p.kv_len)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_evict_by_hand():
    acc = np.array([[[9, 1, 5, 2, 5, 0, 7, 1], [0, 1, 0, 2, 0, 0, 0, 1]]], np.float32)   # totals 9 2 5 4 5 0 7 2
    rows = np.array([[10, 11, 12, 13, 14, -1, 16, 17]], np.int32)
    r, n, a, kept, freed = oracle.evict(acc, rows, None, 1, 1, 2, 5)
    assert kept.tolist() == [[0, 2, 6, 7, -1]] and n.tolist() == [4]      # 6 and, of the tied 2 and 4, the first
    assert r.tolist() == [[10, 12, 16, 17, -1]] and freed.tolist() == [[11, 13, 14] + [-1] * 5]
    assert a[0, 1].tolist() == [0, 0, 0, 1, 0]
    r, n, _, kept, freed = oracle.evict(acc, rows, np.array([3], np.int32), 1, 1, 2, 5)
    assert n.tolist() == [3] and freed.tolist() == [[-1] * 8]


def test_outward_rounding_brackets_and_is_tight():
    g = synth.rng(8)
    x = (g.standard_normal(500) * np.exp(3 * g.standard_normal(500)))
    for fmt in ("bf16", "f16"):
        up, dn = (oracle.widen(oracle.round_outward(x, u, fmt), fmt) for u in (True, False))
        assert (dn <= x).all() and (x <= up).all()
        step = np.abs(x) * (2.0 ** -7 if fmt == "bf16" else 2.0 ** -10) + 2.0 ** -24
        assert (up - dn <= step).all()
        exact = oracle.widen(oracle.round_outward(up, True, fmt), fmt)
        assert np.array_equal(exact, up)


def test_block_scores_bound_every_key_and_are_reached_by_one_key():
    g = synth.rng(5)
    k = g.standard_normal((128, 2, 8))
    q = g.standard_normal((1, 2, 4, 8))
    kmin = np.stack([k[:64].min(0), k[64:].min(0)])
    kmax = np.stack([k[:64].max(0), k[64:].max(0)])
    sc = oracle.block_scores(q, kmin, kmax, np.array([[1, 0, -1]], np.int32), np.array([190], np.int32))
    assert sc.shape == (1, 2, 3) and np.isneginf(sc[0, :, 2]).all()
    for h in range(4):
        for i in range(2):
            d = k[:, h // 2] @ q[0, i, h]
            assert d[64:].max() <= sc[0, h // 2, 0] and d[:64].max() <= sc[0, h // 2, 1]
    one = np.repeat(k[:1], 2, axis=0)     # a block of one key: the bound is the dot product
    sc = oracle.block_scores(q[:, :1], one, one, np.array([[0]], np.int32), np.array([1], np.int32))
    want = [max(k[0, g] @ q[0, 0, h] for h in (2 * g, 2 * g + 1)) for g in range(2)]
    assert np.allclose(sc[0, :, 0], want, rtol=1e-13)


def test_block_rows_by_hand():
    score = np.array([[[0.0, 3.0, np.nan, 3.0, 9.0]]])
    rows, n = oracle.block_rows(score, np.array([[7, 2, 0, 5, 1]], np.int32), np.array([64 * 4 + 3], np.int32), 1, 1, 1, 256)
    want = list(range(448, 512)) + list(range(128, 192)) + [64, 65, 66]
    assert n.tolist() == [[131]] and rows[0, 0, :131].tolist() == want and (rows[0, 0, 131:] == -1).all()
    rows, n = oracle.block_rows(score, np.array([[7, 2, 0, 5, 1]], np.int32), np.array([64 * 4 + 3], np.int32), 0, 0, 2, 128)
    assert n.tolist() == [[67]] and rows[0, 0, 64:67].tolist() == [64, 65, 66]   # blocks 1 and 4: the tie goes to 1


def test_block_scores_use_the_bound_of_each_sign_alone():
    inf = np.inf
    q = np.array([[[[-1.0, 1.0, 0.0]]]])
    table, n = np.array([[0]], np.int32), np.array([64], np.int32)

    def score(lo, hi):
        return oracle.block_scores(q, np.array([[lo]], float), np.array([[hi]], float), table, n)[0, 0, 0]
    assert score([-2, -1, -1], [3, 4, 1]) == 6.0
    assert score([-2, -inf, -inf], [inf, 4, inf]) == 6.0          # bounds that no component uses
    assert score([-inf, -1, -1], [3, 4, 1]) == inf and score([-2, -1, -1], [3, inf, 1]) == inf
    assert score([inf, -1, -1], [inf, 4, 1]) == -inf              # every key infinite where q is negative
    assert np.isnan(score([inf, inf, -1], [inf, inf, 1]))         # -inf and inf meet
    assert np.isnan(score([-2, np.nan, -1], [3, 4, 1])) and np.isnan(score([np.nan, 1, 1], [np.nan, 1, 1]))
    # a key beyond f16 has the bound inf, and none of its products exceeds the score
    k = np.full((64, 1, 3), 0.5)
    k[9, 0, 0] = 127 * 600.0
    lo, hi = (oracle.widen(b, "f16") for b in oracle.block_bounds(k, [0], None, *np.zeros((2, 1, 1, 3), np.uint16), "f16"))
    assert hi[0, 0, 0] == inf
    assert (k[:, 0] @ q[0, 0, 0]).max() <= oracle.block_scores(q, lo, hi, table, n)[0, 0, 0] == 0.0
