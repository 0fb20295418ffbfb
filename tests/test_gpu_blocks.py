"""Block bounds, block scores, block row lists and attention over one list per KV head, against the fp64 oracle."""
import time

import numpy as np
import pytest
import torch

import oracle
import synth
import row_indexed_flash_gb300 as far

from helpers import assert_lse, assert_parity, dev_bits, widen
from test_gpu_weights import QUANT

pytestmark = pytest.mark.gpu


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


# ---------------------------------------------------------------------------
# bounds


def pool(seed, R, Hkv, D, kv, dtype):
    kb = synth.normal_bits(synth.rng(seed), (R, Hkv, D), dtype)
    kd, ks, k64 = dev_bits(kb, dtype), None, widen(kb, dtype)
    if kv in QUANT:
        quant, oq, od = QUANT[kv]
        kd, ks = quant(kd, R)
        k64 = od(*oq(k64.astype(np.float32))).astype(np.float64)
    return kd, ks, k64


@pytest.mark.parametrize("kv", ["bf16", "f16", "i8", "i4", "f8"])
@pytest.mark.parametrize("Hkv,D,dtype", [(8, 128, "bf16"), (2, 64, "f16"), (3, 256, "bf16"), (1, 64, "bf16"), (5, 96, "f16"),
                                         (8, 256, "f16")])
def test_bounds_match_oracle(kv, Hkv, D, dtype):
    dtype = kv if kv in ("bf16", "f16") else dtype
    P = 11
    kd, ks, k64 = pool(60 + D, P * 64, Hkv, D, kv, dtype)
    pages = np.array([7, 0, 10, -1, 3, 11, 5, 2], np.int32)      # -1 and 11 are skipped
    fill = np.array([64, 1, 63, 64, 0, 64, 100, 17], np.int32)   # 0 is skipped, 100 means 64
    start = synth.normal_bits(synth.rng(61), (2, P, Hkv, D), dtype)
    lo, hi = dev_bits(start[0], dtype), dev_bits(start[1], dtype)
    want = oracle.block_bounds(k64, pages, fill, start[0], start[1], dtype)
    got = far.fa_kv_block_bounds(kd, cuda(pages), cuda(fill), lo, hi, k_scale=ks)
    assert got[0] is lo and got[1] is hi
    for g, w in zip(got, want):
        assert np.array_equal(widen(bits(g), dtype), widen(w, dtype))
    full = far.fa_kv_block_bounds(kd, cuda(pages[:1]), None, lo, hi, k_scale=ks)
    assert np.array_equal(widen(bits(full[0])[7], dtype), widen(want[0][7], dtype))


def test_bounds_keep_a_nan_and_ignore_rows_past_the_fill():
    kd, _, _ = pool(62, 128, 2, 64, "bf16", "bf16")
    kd[3, 1, 5] = float("nan")
    kd[64 + 10] = float("nan")
    lo, hi = (torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    far.fa_kv_block_bounds(kd, cuda(np.array([0, 1], np.int32)), cuda(np.array([64, 10], np.int32)), lo, hi)
    for t in (lo, hi):
        bad = torch.isnan(t)
        assert bad.sum() == 1 and bad[0, 1, 5]
    ks = torch.ones((1, 1, 64), dtype=torch.float16, device="cuda")
    ks[0, 0, 9] = float("nan")
    lo, hi = (torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    far.fa_kv_block_bounds(torch.zeros((64, 1, 64), dtype=torch.int8, device="cuda"), cuda(np.array([0], np.int32)), None,
                           lo, hi, k_scale=ks)
    assert torch.isnan(lo).all() and torch.isnan(hi).all()


# ---------------------------------------------------------------------------
# scores: |got - exact| <= (2 D + 2) * 2^-23 * sum |terms| of the best query, at most that of any query


def score_case(seed, S, Nq, Hq, Hkv, D, P, NB, lens, dtype="bf16", slice_seq=None, n_seq=None):
    g = synth.rng(seed)
    n_seq = n_seq or S
    q = synth.normal_bits(g, (S, Nq, Hq, D), dtype)
    a, b = (widen(synth.normal_bits(g, (P, Hkv, D), dtype), dtype) for _ in range(2))
    to = synth.f32_to_bf16_bits if dtype == "bf16" else synth.f32_to_f16_bits
    lo, hi = (to(np.asarray(x, np.float32)) for x in (np.minimum(a, b), np.maximum(a, b)))
    table = np.stack([g.permutation(P)[:NB] for _ in range(n_seq)]).astype(np.int32)
    return q, lo, hi, table, np.asarray(lens, np.int32), None if slice_seq is None else np.asarray(slice_seq, np.int32), dtype


def check_scores(q, lo, hi, table, lens, slice_seq, dtype):
    got = far.fa_kv_block_scores(dev_bits(q, dtype), dev_bits(lo, dtype), dev_bits(hi, dtype), cuda(table), cuda(lens),
                                 slice_seq=cuda(slice_seq), check_status=True).cpu().numpy().astype(np.float64)
    args = [widen(x, dtype) for x in (q, lo, hi)]
    want = oracle.block_scores(*args, table, lens, slice_seq)
    big = oracle.block_scores(np.abs(args[0]), -np.maximum(np.abs(args[1]), np.abs(args[2])),
                              np.maximum(np.abs(args[1]), np.abs(args[2])), table, lens, slice_seq)
    fin = np.isfinite(want)
    assert np.array_equal(fin, np.isfinite(got)) and np.array_equal(np.isneginf(want), np.isneginf(got))
    err = np.abs(got[fin] - want[fin]) - (2 * q.shape[-1] + 2) * 2.0 ** -23 * big[fin]
    assert (err <= 0).all(), err.max()
    return got


@pytest.mark.parametrize("case", [
    dict(S=2, Nq=1, Hq=8, Hkv=2, D=128, P=40, NB=30, lens=[30 * 64, 100]),
    dict(S=3, Nq=1, Hq=4, Hkv=4, D=64, P=9, NB=7, lens=[0, 1, 64 * 7]),
    dict(S=2, Nq=3, Hq=14, Hkv=2, D=256, P=200, NB=131, lens=[65, 64 * 130 + 1], dtype="f16"),
    dict(S=2, Nq=1, Hq=16, Hkv=1, D=128, P=300, NB=300, lens=[300 * 64, 200 * 64 + 5]),
    dict(S=3, Nq=70, Hq=8, Hkv=2, D=128, P=80, NB=70, lens=[64 * 70, 100, 64 * 69 + 2], slice_seq=[0, 0, 1], n_seq=2),
    dict(S=2, Nq=33, Hq=12, Hkv=4, D=64, P=80, NB=20, lens=[1000, 1280], slice_seq=[1, 0], n_seq=2, dtype="f16"),
    dict(S=1, Nq=130, Hq=5, Hkv=1, D=256, P=140, NB=140, lens=[140 * 64 - 63]),
    dict(S=3, Nq=2, Hq=4, Hkv=2, D=64, P=20, NB=10, lens=[640, 640, 640], slice_seq=[0, 5, -1], n_seq=1),   # two with no table
])
def test_scores_match_oracle(case):
    check_scores(*score_case(70 + case["NB"], **case))


def test_scores_skip_bad_pages_and_keep_nan():
    q, lo, hi, table, lens, _, _ = score_case(80, 2, 1, 8, 2, 128, 40, 30, [1920, 1920])
    table[0, 3], table[1, 4] = -1, 40
    got = check_scores(q, lo, hi, table, lens, None, "bf16")
    assert np.isneginf(got[0, :, 3]).all() and np.isneginf(got[1, :, 4]).all()
    hi2 = hi.copy()
    hi2[table[0, 7], 1, 9] = 0x7FC0
    out = far.fa_kv_block_scores(dev_bits(q, "bf16"), dev_bits(lo, "bf16"), dev_bits(hi2, "bf16"), cuda(table), cuda(lens))
    nan = torch.isnan(out).cpu().numpy()
    want = np.zeros_like(nan)
    want[0, 1, 7] = True
    if (table[1] == table[0, 7]).any():
        want[1, 1, list(table[1]).index(table[0, 7])] = True
    assert np.array_equal(nan, want)


def test_scores_bound_the_logits_of_every_key():
    kd, _, k64 = pool(81, 20 * 64, 2, 128, "bf16", "bf16")
    lo, hi = (torch.zeros((20, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    far.fa_kv_block_bounds(kd, torch.arange(20, dtype=torch.int32, device="cuda"), None, lo, hi)
    q = synth.normal_bits(synth.rng(82), (1, 4, 8, 128), "bf16")
    table = np.arange(20, dtype=np.int32)[None]
    sc = far.fa_kv_block_scores(dev_bits(q, "bf16"), lo, hi, cuda(table), cuda(np.array([1280], np.int32))).cpu().numpy()
    dots = np.einsum("rgd,ighd->grih", k64, oracle.widen_bf16(q)[0].reshape(4, 2, 4, 128)).reshape(2, 20, -1).max(-1)
    assert (sc[0] >= dots - 1e-3).all()


# ---------------------------------------------------------------------------
# block rows


@pytest.mark.parametrize("case", [
    dict(S=2, Hkv=3, NB=40, lens=[40 * 64, 100], sinks=1, recent=2, k=5),
    dict(S=3, Hkv=2, NB=7, lens=[0, 1, 448], sinks=0, recent=1, k=0),
    dict(S=2, Hkv=2, NB=300, lens=[64 * 300 - 1, 64 * 299], sinks=2, recent=0, k=50, ties=True),
    dict(S=2, Hkv=1, NB=5000, lens=[320000, 64 * 4100 + 3], sinks=1, recent=3, k=900, ties=True),
    dict(S=4, Hkv=2, NB=33, lens=[2112, 700, 64, 5000], sinks=3, recent=2, k=40),        # all blocks; a length past the table
    dict(S=3, Hkv=2, NB=64, lens=[4000, 4096, 1000], sinks=1, recent=2, k=8, slice_seq=[1, 0, 7], n_seq=2, extra=33),
    dict(S=1, Hkv=1, NB=40000, lens=[40000 * 64], sinks=1, recent=1, k=100),             # past the keys kept on chip
    dict(S=2, Hkv=2, NB=100, lens=[6400, 6399], sinks=0, recent=0, k=3, special=True),
])
def test_block_rows_match_oracle(case):
    g = synth.rng(90 + case["NB"])
    S, Hkv, NB = case["S"], case["Hkv"], case["NB"]
    n_seq = case.get("n_seq", S)
    sc = (g.integers(0, 6, size=(S, Hkv, NB)) if case.get("ties") else g.standard_normal((S, Hkv, NB))).astype(np.float32)
    if case.get("special"):
        sc[g.random(sc.shape) < 0.9] = np.nan
        sc[g.random(sc.shape) < 0.02] = -np.inf
        sc[g.random(sc.shape) < 0.05] = -0.0
        sc[0, 0, -1] = np.inf                             # the last, partial block by score
    table = np.stack([g.permutation(2 * NB)[:NB] for _ in range(n_seq)]).astype(np.int32)
    table[0, NB // 2] = -1
    lens = np.asarray(case["lens"], np.int32)
    seq = None if "slice_seq" not in case else np.asarray(case["slice_seq"], np.int32)
    L = 64 * (case["sinks"] + case["recent"] + case["k"]) + case.get("extra", 0)
    want = oracle.block_rows(sc, table, lens, case["sinks"], case["recent"], case["k"], L, seq)
    got = far.fa_kv_block_rows(cuda(sc), cuda(table), cuda(lens), case["sinks"], case["recent"], case["k"],
                               slice_seq=cuda(seq), list_len=L)
    assert np.array_equal(got[1].cpu().numpy(), want[1])
    assert np.array_equal(got[0].cpu().numpy(), want[0])


# ---------------------------------------------------------------------------
# attention over one list per KV head


def head_lists(seed, S, Hkv, L, R, lens=None, runs=0):
    g = synth.rng(seed)
    rows = np.empty((S, Hkv, L), np.int32)
    for s in range(S):
        for h in range(Hkv):
            if runs:
                start = g.permutation(R // runs)[: -(-L // runs)] * runs
                rows[s, h] = (start[:, None] + np.arange(runs)).reshape(-1)[:L]
            else:
                rows[s, h] = g.permutation(R)[:L]
    return rows, None if lens is None else np.asarray(lens, np.int32)


@pytest.mark.parametrize("kv", ["bf16", "f16", "i8", "i4", "f8"])
@pytest.mark.parametrize("case", [
    dict(S=2, Nq=1, Hq=8, Hkv=2, D=128, L=700, runs=64, lens=[[700, 65], [0, 639]]),
    dict(S=3, Nq=2, Hq=8, Hkv=4, D=128, L=333, causal=True),
    dict(S=1, Nq=1, Hq=16, Hkv=2, D=256, L=2000, runs=64),
    dict(S=2, Nq=1, Hq=4, Hkv=2, D=64, L=260, lens=[[1, 260], [17, 128]]),
    dict(S=1, Nq=4, Hq=16, Hkv=2, D=128, L=6000, runs=64, causal=True, lens=[[6000, 5000]]),
])
def test_decode_heads_match_oracle(kv, case):
    D, R = case["D"], 8192
    if kv in ("i4", "f8") and D != 128:
        pytest.skip("INT4 and FP8 pools are decoded at D 128")
    q = "f16" if kv == "f16" else "bf16"
    kd, ks, k64 = pool(100, R, case["Hkv"], D, kv, q)
    vd, vs, v64 = pool(101, R, case["Hkv"], D, kv, q)
    qb = synth.normal_bits(synth.rng(102), (case["S"], case["Nq"], case["Hq"], D), q)
    rows, lens = head_lists(103, case["S"], case["Hkv"], case["L"], R, case.get("lens"), case.get("runs", 0))
    rows[0, 0, 3] = -1
    rows[-1, -1, 5] = R + 1
    causal = case.get("causal", False)
    kw = dict(kv_len=cuda(lens), causal=causal, k_scale=ks, v_scale=vs, want_lse=True, check_status=True)
    out, lse = far.fa_rows_decode_heads(dev_bits(qb, q), kd, vd, cuda(rows), D ** -0.5, **kw)
    orows = np.where(rows >= R, -1, rows)
    ref, ref_lse = oracle.attend_rows_heads(widen(qb, q), k64, v64, orows, D ** -0.5, causal=causal, kv_len=lens)
    assert_parity(out, ref, "decode heads")
    assert_lse(lse, ref_lse)
    hint = int(rows.size if lens is None else lens.sum()) // case["Hkv"]
    out2, _ = far.fa_rows_decode_heads(dev_bits(qb, q), kd, vd, cuda(rows), D ** -0.5, n_valid_hint=hint, **kw)
    assert_parity(out2, ref, "decode heads, hinted")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", [
    dict(S=2, Nq=128, Hq=8, Hkv=2, L=1000, runs=64, causal=True),
    dict(S=2, Nq=37, Hq=4, Hkv=4, L=300, runs=64, lens=[[300, 40, 0, 128], [64, 65, 299, 127]]),
    dict(S=1, Nq=200, Hq=12, Hkv=4, L=513, causal=True, lens=[[513, 200, 300, 256]]),
    dict(S=1, Nq=64, Hq=8, Hkv=2, L=2048, runs=128, causal=True),
    dict(S=1, Nq=64, Hq=8, Hkv=2, L=2048, runs=64, causal=True, big_v=True),
])
def test_prefill_heads_match_oracle(dtype, case):
    R, D = 4096, 128
    g = synth.rng(110)
    kb, vb = (synth.normal_bits(g, (R, case["Hkv"], D), dtype) for _ in range(2))
    rows, lens = head_lists(111, case["S"], case["Hkv"], case["L"], R, case.get("lens"), case.get("runs", 0))
    if case.get("big_v") and dtype == "bf16":
        # beyond f16's range in head 1's list only, and in a row head 0 alone does not list
        vb[rows[0, 1, 10], 1, 3] = 0x4790
    qb = synth.normal_bits(g, (case["S"], case["Nq"], case["Hq"], D), dtype)
    causal = case.get("causal", False)
    out, lse = far.fa_rows_prefill_heads(dev_bits(qb, dtype), dev_bits(kb, dtype), dev_bits(vb, dtype), cuda(rows), D ** -0.5,
                                         kv_len=cuda(lens), causal=causal, want_lse=True, check_status=True)
    ref, ref_lse = oracle.attend_rows_heads(widen(qb, dtype), kb, vb, rows, D ** -0.5, causal=causal, kv_len=lens, kv_format=dtype)
    if case.get("big_v"):
        assert np.abs(out.cpu().numpy() - ref).max() <= 2e-3 * max(1.0, np.abs(ref).max())
    else:
        assert_parity(out, ref, "prefill heads")
    assert_lse(lse, ref_lse)


def test_head_lists_equal_plain_lists_bit_for_bit():
    p = synth.random_problem(120, S=2, Nq=1, Hq=8, Hkv=2, D=128, R=4096, L=1500, kv_len=True)
    q, k, v = (dev_bits(x, "bf16") for x in (p.q, p.k, p.v))
    rows = torch.from_numpy(p.kv_rows).cuda()
    lens = torch.from_numpy(p.kv_len).cuda()
    a, la = far.fa_rows_decode(q, k, v, rows, p.scale, kv_len=lens, want_lse=True)
    b, lb = far.fa_rows_decode_heads(q, k, v, rows[:, None].repeat(1, 2, 1), p.scale, kv_len=lens[:, None].repeat(1, 2), want_lse=True)
    assert torch.equal(a, b) and torch.equal(la, lb)


# ---------------------------------------------------------------------------
# the operators together


def _cache(seed, n, Hkv, D, dtype="bf16"):
    """A paged sequence of n keys and values: pool tensors, page table, bounds."""
    pages = -(-n // 64)
    g = synth.rng(seed)
    kb, vb = (synth.normal_bits(g, (pages * 64 + 128, Hkv, D), dtype) for _ in range(2))
    table = g.permutation(pages + 2)[:pages].astype(np.int32)[None]
    kd, vd = dev_bits(kb, dtype), dev_bits(vb, dtype)
    lo, hi = (torch.zeros((pages + 2, Hkv, D), dtype=kd.dtype, device="cuda") for _ in range(2))
    fill = np.full(pages, 64, np.int32)
    fill[-1] = n - 64 * (pages - 1)
    far.fa_kv_block_bounds(kd, cuda(table[0]), cuda(fill), lo, hi)
    return kb, vb, kd, vd, table, lo, hi


def test_block_sparse_decode_chain():
    n, Hq, Hkv, D = 3000, 8, 2, 128
    kb, vb, kd, vd, table, lo, hi = _cache(130, n, Hkv, D)
    qb = synth.normal_bits(synth.rng(131), (1, 1, Hq, D), "bf16")
    lens = np.array([n], np.int32)
    sc = far.fa_kv_block_scores(dev_bits(qb, "bf16"), lo, hi, cuda(table), cuda(lens))
    rows, ln = far.fa_kv_block_rows(sc, cuda(table), cuda(lens), 1, 2, 9)
    want = oracle.block_rows(sc.cpu().numpy(), table, lens, 1, 2, 9, 12 * 64)
    assert np.array_equal(rows.cpu().numpy(), want[0]) and np.array_equal(ln.cpu().numpy(), want[1])
    out, _ = far.fa_rows_decode_heads(dev_bits(qb, "bf16"), kd, vd, rows, D ** -0.5, kv_len=ln)
    ref, _ = oracle.attend_rows_heads(oracle.widen_bf16(qb), kb, vb, want[0], D ** -0.5, kv_len=want[1], kv_format="bf16")
    assert_parity(out, ref, "chain")
    # with every block chosen it is the attention over the whole sequence
    rows, ln = far.fa_kv_block_rows(sc, cuda(table), cuda(lens), 1, 2, 44)
    out, lse = far.fa_rows_decode_heads(dev_bits(qb, "bf16"), kd, vd, rows, D ** -0.5, kv_len=ln, want_lse=True)
    full = far.fa_kv_page_table_to_rows(cuda(table), cuda(lens), 47 * 64)
    ref, lref = far.fa_rows_decode(dev_bits(qb, "bf16"), kd, vd, full, D ** -0.5, kv_len=cuda(lens), want_lse=True)
    assert (out - ref).abs().max() <= 1e-4 and (lse - lref).abs().max() <= 1e-4


def test_block_sparse_prompt_chain_in_a_graph():
    n, Nq, Hq, Hkv, D = 2000, 128, 8, 2, 128
    kb, vb, kd, vd, table, lo, hi = _cache(140, n, Hkv, D)
    S = 3                                                     # three tiles of 128 queries of one sequence
    qb = synth.normal_bits(synth.rng(141), (S, Nq, Hq, D), "bf16")
    lens = np.array([n - 256, n - 128, n], np.int32)
    seq = torch.zeros(S, dtype=torch.int32, device="cuda")
    q, tb, ln = dev_bits(qb, "bf16"), cuda(table), cuda(lens)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def chain():
        sc = far.fa_kv_block_scores(q, lo, hi, tb, ln, slice_seq=seq, workspace=ws)
        rows, m = far.fa_kv_block_rows(sc, tb, ln, 1, 3, 8, slice_seq=seq)
        out, lse = far.fa_rows_prefill_heads(q, kd, vd, rows, D ** -0.5, kv_len=m, causal=True, want_lse=True, workspace=ws)
        return sc, rows, m, out, lse

    first = chain()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = chain()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    sc, rows, m, out, lse = first
    want = oracle.block_rows(sc.cpu().numpy(), table, lens, 1, 3, 8, 12 * 64, np.zeros(S, np.int32))
    assert np.array_equal(rows.cpu().numpy(), want[0])
    pick = [0, 1, 63, 127]
    ref, lref = oracle.attend_rows_heads(oracle.widen_bf16(qb[:, pick]), kb, vb, want[0], D ** -0.5, kv_len=want[1], causal=True,
                                         query_rows=pick, n_query=Nq, kv_format="bf16")
    assert_parity(out[:, pick], ref, "prompt chain")
    assert_lse(lse[:, pick], lref)


def test_scores_of_many_slices_of_alternating_sequences():
    # a CTA walks several slices and stages the bounds again at every change of sequence; one query
    # tile per slice, so the issuing warps take turns
    for Nq, S in ((33, 40), (70, 33), (17, 60)):
        g = synth.rng(150 + Nq)
        seq = g.integers(0, 3, size=S)
        lens = g.integers(0, 64 * 130, size=S)
        lens[::9] = 0
        check_scores(*score_case(151 + Nq, S=S, Nq=Nq, Hq=8, Hkv=2, D=128, P=140, NB=130, lens=lens, slice_seq=seq, n_seq=3))


@pytest.mark.parametrize("D, Nq", [(64, 1), (128, 1), (256, 1), (128, 70), (256, 70)])
def test_scores_are_not_biased_low(D, Nq):
    """Terms of one sign: a running sum that is cut off, not rounded, ends low.

    A step of 16 products cuts off less than 2^-23 of the sum so far; over n equal steps that is
    (n + 1) / 2 * 2^-23 of the result.  One accumulator takes both products up to D 128 (D / 8 steps),
    two take 16 steps each at D 256; one fp32 addition more rounds by 2^-24.
    """
    g = synth.rng(90 + D + Nq)
    q = synth.normal_bits(g, (1, Nq, 8, D), "f16")
    size = [np.abs(widen(synth.normal_bits(g, (150, 2, D), "f16"), "f16")) + 1 for _ in range(2)]
    lo, hi = (synth.f32_to_f16_bits(np.asarray(x, np.float32)) for x in (-size[0], size[1]))
    table, lens = np.arange(150, dtype=np.int32)[None], np.asarray([150 * 64], np.int32)
    got = check_scores(q, lo, hi, table, lens, None, "f16")
    want = oracle.block_scores(widen(q, "f16"), widen(lo, "f16"), widen(hi, "f16"), table, lens, None)
    steps = min(D // 8, 16)
    assert abs(((got - want) / want).mean()) < ((steps + 1) / 2 * 2.0 + 1) * 2.0 ** -24


def test_scores_report_an_expired_wait_and_recover():
    """Every wait of the prompt form runs out in turn, in CTAs that stage the bounds of several sequences."""
    g = synth.rng(170)
    S = 60
    q, lo, hi, table, lens, seq, _ = score_case(171, S=S, Nq=17, Hq=32, Hkv=8, D=128, P=140, NB=130,
                                                lens=g.integers(64, 64 * 130, size=S), slice_seq=np.arange(S) % 3, n_seq=3)
    q, lo, hi = (dev_bits(x, "bf16") for x in (q, lo, hi))
    table, lens, seq = cuda(table), cuda(lens), cuda(seq)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    want = far.fa_kv_block_scores(q, lo, hi, table, lens, slice_seq=seq, workspace=ws, check_status=True)
    try:
        for limit in (1, 1000, 4000, 16000):
            far.fa_set_wait_limit_ns(limit)
            far.fa_kv_block_scores(q, lo, hi, table, lens, slice_seq=seq, workspace=ws)
            assert far.fa_rows_status(ws, clear=True) & far.FA_WS_WAIT_EXPIRED or limit > 1
    finally:
        far.fa_set_wait_limit_ns(0)
    assert torch.equal(far.fa_kv_block_scores(q, lo, hi, table, lens, slice_seq=seq, workspace=ws, check_status=True), want)


@pytest.mark.parametrize("D,together", [(128, True), (128, False), (256, True), (64, True)])
def test_scores_of_one_token_drain_after_an_expired_wait(D, together):
    """The streaming form, with tile copies (tables of consecutive pages) and with gathers."""
    q, lo, hi, table, lens, _, _ = score_case(180 + D, S=5, Nq=1, Hq=8, Hkv=2, D=D, P=6000, NB=1100, lens=[1100 * 64] * 5)
    if together:
        table[:] = np.arange(1100) + 1000 * np.arange(5)[:, None] - 300 * (np.arange(5)[:, None] > 3)
        table[:, 300:700:130] = 7                        # pages that break some of the runs
    q, lo, hi = (dev_bits(x, "bf16") for x in (q, lo, hi))
    table, lens = cuda(table), cuda(lens)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    want = far.fa_kv_block_scores(q, lo, hi, table, lens, workspace=ws, check_status=True)
    spent = []
    try:
        for limit in (1, 1, 300, 1000, 3000):
            far.fa_set_wait_limit_ns(limit)
            begun = time.monotonic()
            far.fa_kv_block_scores(q, lo, hi, table, lens, workspace=ws)
            assert far.fa_rows_status(ws, clear=True) & far.FA_WS_WAIT_EXPIRED or limit > 1
            spent.append(time.monotonic() - begun)
    finally:
        far.fa_set_wait_limit_ns(0)
    assert torch.equal(far.fa_kv_block_scores(q, lo, hi, table, lens, workspace=ws, check_status=True), want)
    assert max(spent) < 0.5, spent


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Nq", [1, 17, 70])
def test_scores_of_infinite_bounds(D, Nq, dtype):
    """One end or both infinite in some pages, under queries of either sign and zero there."""
    q, lo, hi, table, lens, _, _ = score_case(190 + D + Nq, 2, Nq, 8, 2, D, 200, 140, [140 * 64, 139 * 64 - 5], dtype=dtype)
    inf = 0x7F80 if dtype == "bf16" else 0x7C00
    q[:, :, :, 3] |= 0x8000              # negative
    q[:, :, :, 5] &= 0x7FFF              # positive
    q[:, :, :, 7] = 0
    q[:, 0, 0, 7] = 0x8000               # -0
    hi[0:60, 0, 3] = inf                 # not used: a number
    lo[20:80, 1, 5] = inf | 0x8000       # not used
    lo[90:95, :, 7] = inf | 0x8000       # zeros alone
    hi[90:95, :, 7] = inf
    hi[100:110, 0, 5] = inf              # plus infinity
    lo[110:120, 1, 3] = inf | 0x8000     # plus infinity
    hi[120:124, :, 11] = inf             # as the query's sign there goes
    lo[124:128, :, D - 1] = inf | 0x8000
    lo[128, :, 5] = hi[128, :, 5] = inf | 0x8000   # minus infinity
    table[0, :129] = np.arange(129)
    table[1, :129] = np.arange(129)[::-1]
    got = far.fa_kv_block_scores(dev_bits(q, dtype), dev_bits(lo, dtype), dev_bits(hi, dtype), cuda(table), cuda(lens),
                                 check_status=True).cpu().numpy().astype(np.float64)
    args = [widen(x, dtype) for x in (q, lo, hi)]
    with np.errstate(invalid="ignore"):
        want = oracle.block_scores(*args, table, lens)
    assert not np.isnan(want).any() and np.isfinite(want[0, 0, :60]).all() and np.isposinf(want[0, 0, 100:110]).all()
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin])
    # |got - want| as for finite bounds: the sum of the terms' magnitudes, those of an unused infinite bound left out
    a = [np.where(np.isfinite(x), x, 0.0) for x in args]
    m = np.maximum(np.abs(a[1]), np.abs(a[2]))
    big = oracle.block_scores(np.abs(a[0]), -m, m, table, lens)
    assert (np.abs(got[fin] - want[fin]) <= (2 * D + 2) * 2.0 ** -23 * big[fin]).all()


@pytest.mark.parametrize("Nq", [1, 40])
def test_scores_of_a_mixture_of_nan_and_infinite_bounds(Nq):
    q, lo, hi, table, lens, _, _ = score_case(200 + Nq, 1, Nq, 8, 2, 128, 140, 140, [140 * 64])
    table[0] = np.arange(140)
    lo[5, 0, 9] = hi[5, 0, 9] = 0x7FC0
    lo[6, 1, 9] = 0x7FC0                            # a NaN in one bound is enough, whatever the query's sign
    hi[7, :, 4], lo[8, :, 4] = 0x7F80, 0xFF80
    q[0, -1, 2, 20] = 0x7FC0                        # a NaN query vector of head 2: KV head 0
    args = [widen(x, "bf16") for x in (q, lo, hi)]
    with np.errstate(invalid="ignore"):
        want = oracle.block_scores(*args, table, lens)
    got = far.fa_kv_block_scores(dev_bits(q, "bf16"), dev_bits(lo, "bf16"), dev_bits(hi, "bf16"), cuda(table), cuda(lens),
                                 check_status=True).cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(want[0, 0]).all() and np.isnan(want[0, 1, 6])
    fin = ~np.isnan(want)
    assert np.array_equal(np.isinf(got[fin]), np.isinf(want[fin]))


def test_a_block_with_a_key_beyond_f16_is_chosen():
    # INT8 codes whose value passes 65504: the f16 bound is infinite, and a query that points away from
    # that key still ranks the block by its other keys
    P, D = 12, 64
    kd = torch.ones((P * 64, 1, D), dtype=torch.int8, device="cuda")
    ks = torch.full((P, 1, 64), 0.25, dtype=torch.float16, device="cuda")
    kd[5 * 64 + 3, 0, 0], ks[5, 0, 3] = 127, 600.0
    kd[5 * 64 + 9, 0, 1] = 100
    pages = torch.arange(P, dtype=torch.int32, device="cuda")
    lo, hi = (torch.zeros((P, 1, D), dtype=torch.float16, device="cuda") for _ in range(2))
    far.fa_kv_block_bounds(kd, pages, None, lo, hi, k_scale=ks)
    assert torch.isposinf(hi[5, 0, 0]) and torch.isfinite(lo).all()
    q = torch.zeros((1, 1, 1, D), dtype=torch.float16, device="cuda")
    q[0, 0, 0, 0], q[0, 0, 0, 1] = -1.0, 1.0
    n = torch.tensor([P * 64], dtype=torch.int32, device="cuda")
    sc = far.fa_kv_block_scores(q, lo, hi, pages[None], n)
    assert sc[0, 0, 5] == 600.0 - 0.25 and (sc[0, 0, :5] == 0).all()
    rows, _ = far.fa_kv_block_rows(sc, pages[None], n, 0, 0, 1)
    assert rows[0, 0, 0] == 5 * 64


def test_current_stream_is_the_same_by_both_interfaces(monkeypatch):
    side = torch.cuda.Stream()
    dev = torch.device("cuda", torch.cuda.current_device())
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            fast = far._stream(None, dev)
            with monkeypatch.context() as m:
                m.setattr(far, "_raw_stream", None)
                assert far._stream(None, dev) == fast == stream.cuda_stream
