"""Accumulated attention weight (fa_rows_weights) against the fp64 oracle.

Bound, per accumulated entry: a term exp(x - lse) has an exponent error of at
most e = (D + 8) * 2^-23 * scale * sum_d |q_d k_d| + 2^-22 * (|x| + |lse| + 1)
(the fp32 dot product of exact products, its scaling, and the base-2 argument;
2^-23 a step, since the tensor core's sums need not round to nearest), the
hardware exponential 2^-21, and the sum of nv terms nv * 2^-24 of itself.
"""
import ctypes
import threading
import time

import numpy as np
import pytest
import torch

import oracle
import synth
import row_indexed_flash_gb300 as far

from helpers import dev_bits, widen

pytestmark = pytest.mark.gpu

QUANT = {"i8": (far.fa_kv_quantize_int8, oracle.quantize_int8, oracle.dequantize_int8),
         "i4": (far.fa_kv_quantize_int4, oracle.quantize_int4, oracle.dequantize_int4),
         "f8": (far.fa_kv_quantize_fp8, oracle.quantize_fp8, oracle.dequantize_fp8)}


def make(seed, kv="bf16", q="bf16", **kw):
    """(problem, device K and scales, fp64 K) of one random problem."""
    p = synth.random_problem(seed, dtype=q, **kw)
    kd = dev_bits(p.k, q)
    k64 = widen(p.k, q)
    if kv in QUANT:
        quant, oq, od = QUANT[kv]
        kd, ks = quant(kd, p.R)
        k64 = od(*oq(k64.astype(np.float32))).astype(np.float64)
    else:
        ks = None
    return p, kd, ks, k64


def lse_of(p, k64):
    """fp32 log-sum-exp, as an attention call returns it."""
    _, lse = oracle.attend_rows(widen(p.q, p.dtype), k64, np.zeros_like(k64), p.kv_rows, p.scale,
                                mask=None if p.mask is None else p.mask.astype(np.float64), causal=p.causal,
                                kv_len=p.kv_len)
    return lse.astype(np.float32)


def bound(p, k64, lse, w):
    q = widen(p.q, p.dtype)
    G = p.Hq // p.Hkv
    rows = np.clip(p.kv_rows, 0, p.R - 1).astype(np.int64)
    fin = np.where(np.isfinite(lse), lse, 0.0).astype(np.float64)
    worst = np.zeros_like(w)
    for s in range(p.S):
        for g in range(p.Hkv):
            k = k64[rows[s], g]
            qq = q[s, :, g * G:(g + 1) * G].reshape(-1, p.D)
            x = np.abs(p.scale * (k @ qq.T)) + (np.abs(p.mask[s]).T.repeat(G, 1) if p.mask is not None else 0.0)
            x = np.where(np.isfinite(x), x, 0.0)
            e = (p.D + 8) * 2.0 ** -23 * abs(p.scale) * (np.abs(k) @ np.abs(qq).T) + 2.0 ** -22 * (
                x + np.abs(fin[s, :, g * G:(g + 1) * G]).reshape(1, -1) + 1.0)
            worst[s, g] = e.max(axis=1)
    return w * (np.expm1(worst) + 2.0 ** -21 + p.Nq * G * 2.0 ** -24) + 1e-35


def run(p, kd, ks, lse, acc=None, **kw):
    t = lambda a: None if a is None else torch.from_numpy(a).cuda()
    return far.fa_rows_weights(dev_bits(p.q, p.dtype), kd, t(p.kv_rows), p.scale, t(lse), acc, kv_len=t(p.kv_len),
                               mask=t(p.mask), causal=p.causal, k_scale=ks, check_status=True, **kw)


def check(p, kd, ks, k64, lse=None):
    lse = lse_of(p, k64) if lse is None else lse
    w = oracle.attention_weights(widen(p.q, p.dtype), k64, p.kv_rows, p.scale, lse.astype(np.float64), mask=p.mask,
                                 causal=p.causal, kv_len=p.kv_len)
    got = run(p, kd, ks, lse).cpu().numpy().astype(np.float64)
    err = np.abs(got - w) - bound(p, k64, lse, w)
    assert (err <= 0).all(), (err.max(), np.unravel_index(err.argmax(), err.shape))
    return got


CASES = [
    dict(S=2, Nq=1, Hq=8, Hkv=2, D=128, R=512, L=300),
    dict(S=3, Nq=1, Hq=4, Hkv=4, D=64, R=512, L=1),
    dict(S=1, Nq=1, Hq=16, Hkv=2, D=256, R=512, L=257),
    dict(S=2, Nq=5, Hq=6, Hkv=2, D=128, R=1024, L=700, causal=True, kv_len=True),
    dict(S=2, Nq=3, Hq=14, Hkv=2, D=64, R=640, L=129, causal=True),
    dict(S=1, Nq=65, Hq=8, Hkv=2, D=128, R=2048, L=1111, causal=True, kv_len=True),
    dict(S=2, Nq=129, Hq=4, Hkv=1, D=256, R=1024, L=383, causal=True),
    dict(S=1, Nq=300, Hq=12, Hkv=4, D=128, R=1024, L=640, causal=True, pad_frac=0.0),
    dict(S=1, Nq=40, Hq=16, Hkv=1, D=64, R=1024, L=200),
    dict(S=2, Nq=7, Hq=5, Hkv=5, D=32, R=512, L=100, causal=True),
    dict(S=1, Nq=2, Hq=4, Hkv=2, D=96, R=512, L=130),
    dict(S=2, Nq=4, Hq=8, Hkv=2, D=128, R=512, L=150, with_mask=True, neg_inf_frac=0.3),
    dict(S=2, Nq=20, Hq=8, Hkv=2, D=128, R=512, L=10, causal=True),          # more queries than entries
    dict(S=2, Nq=1, Hq=8, Hkv=2, D=128, R=512, L=200, distinct=False),       # the same row twice
]


@pytest.mark.parametrize("kv", ["bf16", "f16", "i8", "i4", "f8"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_weights_match_oracle(case, kv):
    q = "f16" if kv == "f16" or (kv in QUANT and case % 2) else "bf16"
    check(*make(200 + case, kv, q, **CASES[case]))


def test_weights_of_an_attention_call_sum_to_its_queries():
    p, kd, _, _ = make(31, S=2, Nq=6, Hq=8, Hkv=2, D=128, R=4096, L=3000, causal=True, pad_frac=0.0)
    q, v = dev_bits(p.q, "bf16"), dev_bits(p.v, "bf16")
    rows = torch.from_numpy(p.kv_rows).cuda()
    _, lse = far.fa_rows_prefill(q, kd, v, rows, p.scale, causal=True, want_lse=True)
    acc = far.fa_rows_weights(q, kd, rows, p.scale, lse, causal=True)
    assert torch.allclose(acc.double().sum(2), torch.full((2, 2), 24.0, dtype=torch.float64, device="cuda"), atol=24 * 1e-4)


def test_weights_accumulate_decay_and_leave_the_rest():
    p, kd, ks, k64 = make(32, S=2, Nq=1, Hq=8, Hkv=2, D=128, R=512, L=300, kv_len=True)
    p.kv_len[:] = [0, 123]
    lse = lse_of(p, k64)
    once = run(p, kd, ks, lse)
    assert (once[0] == 0).all() and (once[1, :, 123:] == 0).all()
    start = torch.rand_like(once) + 0.5
    acc = start.clone()
    assert run(p, kd, ks, lse, acc) is acc
    assert torch.equal(acc[0], start[0]) and torch.equal(acc[1, :, 123:], start[1, :, 123:])
    assert torch.allclose(acc[1, :, :123], start[1, :, :123] + once[1, :, :123], rtol=2.0 ** -23, atol=0)
    half = run(p, kd, ks, lse, start.clone(), decay=0.5)
    assert torch.allclose(half[1, :, :123], 0.5 * start[1, :, :123] + once[1, :, :123], rtol=2.0 ** -23, atol=0)
    nan = run(p, kd, ks, lse, torch.full_like(start, float("nan")), decay=0.0)
    assert torch.equal(nan[1, :, :123], once[1, :, :123]) and torch.isnan(nan[0]).all()


@pytest.mark.parametrize("Nq", [1, 70])
def test_weights_of_hidden_queries_rows_and_poison(Nq):
    p, kd, ks, k64 = make(33, S=2, Nq=Nq, Hq=8, Hkv=2, D=128, R=512, L=200, causal=True, pad_frac=0.2)
    lse = lse_of(p, k64)
    lse[0, 0] = -np.inf                       # a query that saw nothing adds nothing
    p.kv_rows[1, 50] = p.R + 7                # out of range: skipped like padding
    clean = check(p, kd, ks, k64, lse)
    assert (clean[1, :, 50] == 0).all()
    unlisted = np.setdiff1d(np.arange(p.R), p.kv_rows)
    kd[torch.from_numpy(unlisted).cuda()] = float("nan")
    assert np.array_equal(run(p, kd, ks, lse).cpu().numpy(), clean.astype(np.float32))
    # a NaN key spoils its own entry only, where some query sees it
    hit = int(np.argmax(p.kv_rows[0] >= 0))
    kd[int(p.kv_rows[0, hit])] = float("nan")
    got = run(p, kd, ks, lse).cpu().numpy()
    same = np.ones(p.L, bool)
    same[hit] = False
    assert np.array_equal(got[0][:, same], clean[0][:, same].astype(np.float32))


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_nan_keys_that_the_causal_limit_hides_add_nothing(kv):
    p, kd, ks, k64 = make(34, kv, S=1, Nq=8, Hq=8, Hkv=2, D=128, R=512, L=8, causal=True, pad_frac=0.0)
    lse = lse_of(p, k64)
    lse[0, -1] = -np.inf                      # the only query that sees the last entry
    last = int(p.kv_rows[0, -1])
    if kv == "bf16":
        kd[last] = float("nan")
    else:
        ks[last // 64, :, last % 64] = float("nan")
    got = run(p, kd, ks, lse)
    assert (got[:, :, -1] == 0).all() and torch.isfinite(got).all()


def test_weights_with_a_mask_of_minus_infinity_over_nan():
    p, kd, ks, k64 = make(35, S=1, Nq=2, Hq=4, Hkv=2, D=128, R=512, L=64, with_mask=True)
    p.mask[0, :, 5] = -np.inf
    lse = lse_of(p, k64)
    p.kv_rows[0, 5] = np.setdiff1d(np.arange(p.R), p.kv_rows)[0]
    kd[int(p.kv_rows[0, 5])] = float("nan")
    got = run(p, kd, ks, lse)
    assert (got[0, :, 5] == 0).all() and torch.isfinite(got).all()


def test_weights_repeat_bit_for_bit_on_streams_and_in_graphs():
    p, kd, ks, k64 = make(36, S=2, Nq=2, Hq=8, Hkv=2, D=128, R=4096, L=3000)
    lse = torch.from_numpy(lse_of(p, k64)).cuda()
    q, rows = dev_bits(p.q, "bf16"), torch.from_numpy(p.kv_rows).cuda()
    want = far.fa_rows_weights(q, kd, rows, p.scale, lse)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        got = far.fa_rows_weights(q, kd, rows, p.scale, lse)
    torch.cuda.current_stream().wait_stream(other)
    assert torch.equal(got, want)
    acc = torch.zeros_like(want)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    far.fa_rows_weights(q, kd, rows, p.scale, lse, acc, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        far.fa_rows_weights(q, kd, rows, p.scale, lse, acc, workspace=ws)
    acc.zero_()
    graph.replay()
    assert torch.equal(acc, want)
    graph.replay()
    assert torch.equal(acc, want + want)


def test_weights_read_pool_rows_past_two_gigabytes():
    R, Hkv, D = (1 << 21) + 64 * 300, 8, 128
    kd = torch.zeros((R, Hkv, D), dtype=torch.int8, device="cuda")
    ks = torch.ones((R // 64, Hkv, 64), dtype=torch.float16, device="cuda")
    rows = torch.tensor([[0, 1, R - 1, R - 2, R, -1]], dtype=torch.int32, device="cuda")
    kd[R - 1] = 1
    kd[1] = 2
    q = torch.ones((1, 1, 16, D), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((1, 1, 16), dtype=torch.float32, device="cuda")
    got = far.fa_rows_weights(q, kd, rows, 1.0 / 128, lse, k_scale=ks, check_status=True)[0]
    want = 2.0 * np.exp([0.0, 2.0, 1.0, 0.0])
    assert np.allclose(got[:, :4].cpu().numpy(), np.tile(want, (8, 1)), rtol=2.0 ** -18) and (got[:, 4:] == 0).all()


def paged_rows(seed, S, L, R, run):
    """Lists of whole runs of `run` consecutive rows in random order, the last one cut."""
    g = synth.rng(seed)
    starts = np.stack([g.permutation(R // run)[: -(-L // run)] * run for _ in range(S)])
    return (starts[:, :, None] + np.arange(run)).reshape(S, -1)[:, :L].astype(np.int32)


@pytest.mark.parametrize("kv", ["bf16", "f16", "i8", "i4", "f8"])
@pytest.mark.parametrize("case", [
    dict(S=3, Nq=1, Hq=8, Hkv=2, D=128, L=5000, run=64, lens=[5000, 63, 4097]),
    dict(S=2, Nq=2, Hq=16, Hkv=2, D=64, L=9000, run=128, lens=[9000, 8191]),
    dict(S=2, Nq=4, Hq=8, Hkv=1, D=256, L=3000, run=64, lens=[1, 3000]),
    dict(S=2, Nq=100, Hq=8, Hkv=2, D=128, L=3000, run=64, lens=[2999, 1500]),
])
def test_weights_over_pages(case, kv):
    c = dict(case)
    run_rows, lens = c.pop("run"), c.pop("lens")
    p, kd, ks, k64 = make(300 + c["L"], kv, "f16" if kv == "f16" else "bf16", R=16384, causal=True, pad_frac=0.0, **c)
    p.kv_rows = paged_rows(301, c["S"], c["L"], 16384, run_rows)
    p.kv_len = np.asarray(lens, np.int32)
    p.kv_rows[0, 2] = -1                      # a hole in a page
    check(p, kd, ks, k64)


def test_weights_of_many_short_slices():
    # more slices than threads of a block, some empty, every share crossing many of them
    S = 1100
    p, kd, ks, k64 = make(320, S=S, Nq=1, Hq=2, Hkv=2, D=64, R=1024, L=140)
    p.kv_len = synth.rng(321).integers(0, 141, size=S).astype(np.int32)
    p.kv_len[::7] = 0
    check(p, kd, ks, k64)


@pytest.mark.parametrize("kv,Nq", [("bf16", 1), ("i8", 1), ("bf16", 40)])
def test_weights_report_an_expired_wait_and_recover(kv, Nq):
    p, kd, ks, k64 = make(330, kv, S=2, Nq=Nq, Hq=8, Hkv=2, D=128, R=8192, L=6000)
    lse = torch.zeros((2, Nq, 8), dtype=torch.float32, device="cuda")
    q, rows = dev_bits(p.q, "bf16"), torch.from_numpy(p.kv_rows).cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    want = far.fa_rows_weights(q, kd, rows, p.scale, lse, k_scale=ks, workspace=ws, check_status=True)
    far.fa_set_wait_limit_ns(1)
    try:
        far.fa_rows_weights(q, kd, rows, p.scale, lse, k_scale=ks, workspace=ws)
        assert far.fa_rows_status(ws, clear=True) & far.FA_WS_WAIT_EXPIRED
    finally:
        far.fa_set_wait_limit_ns(0)
    assert torch.equal(far.fa_rows_weights(q, kd, rows, p.scale, lse, k_scale=ks, workspace=ws, check_status=True), want)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("L", [5, 128, 129])
def test_weights_of_one_tile_slices(kv, L):
    # every (slice, KV head) is one or two tiles: the query buffers change with nearly every tile
    p, kd, ks, k64 = make(340 + L, kv, S=90, Nq=1, Hq=8, Hkv=8, D=128, R=1024, L=L)
    p.kv_len = synth.rng(341).integers(0, L + 1, size=90).astype(np.int32)
    p.kv_len[5:20] = 0
    for _ in range(3):
        check(p, kd, ks, k64)


@pytest.mark.parametrize("kv", ["bf16", "f8"])
@pytest.mark.parametrize("Nq,L,G", [(1500, 1700, 4), (900, 900, 1), (700, 3000, 7), (2048, 2500, 2), (2048, 16384, 4)])
def test_weights_of_long_prompts(kv, Nq, L, G):
    # many query tiles per key tile, key tiles that only late queries see
    p, kd, ks, k64 = make(350 + Nq, kv, S=1, Nq=Nq, Hq=2 * G, Hkv=2, D=128, R=32768, L=L, causal=True, pad_frac=0.02)
    q = dev_bits(p.q, p.dtype).double().view(Nq, 2, G, 128)
    k = torch.from_numpy(k64[np.maximum(p.kv_rows[0], 0)]).cuda()                      # [L, 2, D]
    x = p.scale * torch.einsum("ighd,jgd->gihj", q, k)
    j, i = torch.arange(L, device="cuda"), torch.arange(Nq, device="cuda")
    see = (j[None] <= L - Nq + i[:, None]) & (torch.from_numpy(p.kv_rows[0]).cuda() >= 0)[None]
    x.masked_fill_(~see[None, :, None], -float("inf"))
    lse = torch.logsumexp(x, -1)                                                       # [2, Nq, G]
    want = torch.exp(x - lse[..., None]).nan_to_num(0.0).sum((1, 2))
    lse32 = lse.permute(1, 0, 2).reshape(1, Nq, 2 * G).float().contiguous()
    for _ in range(2):
        got = far.fa_rows_weights(dev_bits(p.q, p.dtype), kd, torch.from_numpy(p.kv_rows).cuda(), p.scale, lse32, causal=True,
                                  k_scale=ks, check_status=True)[0].double()
        # each term: exponent error below 2^-23 * ((D + 8) * 8 + 60) ~ 1.4e-4 for |scale q k| sums below 8, |x| + |lse| below 30
        assert ((got - want).abs() <= 1.4e-4 * want + 1e-35).all(), ((got - want).abs() / want.clamp(min=1e-30)).max()


@pytest.mark.parametrize("Nq,G,L", [(1, 4, 6000), (1, 4, 700), (40, 4, 6000), (40, 4, 130), (70, 1, 3000)])
def test_an_expired_wait_leaves_no_copy_behind(Nq, G, L):
    """Lists of whole pages (tile copies) with shuffled ones between (gathers), few tiles and many.

    A call whose waits run out drains its own copies before it ends: that takes microseconds, not the second
    after which a drain gives up, as it would if it waited for a warp that had left.
    """
    p, kd, _, _ = make(360 + L + Nq, "bf16", S=2, Nq=Nq, Hq=2 * G, Hkv=2, D=128, R=16384, L=L)
    rows = paged_rows(361, 2, -(-L // 64) * 64, 16384, 64).reshape(2, -1, 64)
    rows[:, 2::3] = rows[:, 2::3, ::-1]
    rows = torch.from_numpy(np.ascontiguousarray(rows.reshape(2, -1)[:, :L])).cuda()
    lse = torch.zeros((2, Nq, 2 * G), dtype=torch.float32, device="cuda")
    q = dev_bits(p.q, "bf16")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    want = far.fa_rows_weights(q, kd, rows, p.scale, lse, workspace=ws, check_status=True)
    spent = []
    try:
        for limit in (1, 1, 300, 1000, 3000):
            far.fa_set_wait_limit_ns(limit)
            begun = time.monotonic()
            far.fa_rows_weights(q, kd, rows, p.scale, lse, workspace=ws)
            assert far.fa_rows_status(ws, clear=True) & far.FA_WS_WAIT_EXPIRED or limit > 1
            spent.append(time.monotonic() - begun)
    finally:
        far.fa_set_wait_limit_ns(0)
    assert torch.equal(far.fa_rows_weights(q, kd, rows, p.scale, lse, workspace=ws, check_status=True), want)
    assert max(spent) < 0.5, spent


def test_weights_of_several_head_dims_from_several_threads():
    """Calls of one kernel that need unequal amounts of shared memory, at the same time."""
    cases = []
    for D in (256, 96, 32, 224):
        p, kd, _, _ = make(380 + D, S=1, Nq=2, Hq=4, Hkv=2, D=D, R=512, L=130, with_mask=True)
        q, rows, mask = dev_bits(p.q, "bf16"), torch.from_numpy(p.kv_rows).cuda(), torch.from_numpy(p.mask).cuda()
        lse = torch.zeros((1, 2, 4), device="cuda")
        acc, ws = torch.zeros((1, 2, 130), device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()
        want = far.fa_rows_weights(q, kd, rows, 0.05, lse, mask=mask, decay=0.0)
        a, out, _ = far.make_args(q, kd, kd, rows, 0.05, mask=mask)
        args = (ctypes.byref(a), lse.data_ptr(), 0.0, acc.data_ptr(), ws.data_ptr(), 256, stream.cuda_stream)
        cases.append((D, args, acc, want, (q, kd, rows, mask, lse, ws, out, a, stream)))
    torch.cuda.synchronize()
    call, wrong = far.lib().fa_rows_weights, []

    def work(D, args):
        for _ in range(4000):
            if call(*args):
                wrong.append((D, far.fa_last_error()))
                return

    threads = [threading.Thread(target=work, args=c[:2], daemon=True) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=60)
        assert not t.is_alive()
    torch.cuda.synchronize()
    assert not wrong, wrong[:3]
    for D, _, acc, want, _ in cases:
        assert torch.equal(acc, want), D


@pytest.mark.parametrize("kv,dtype", [("bf16", "bf16"), ("f16", "f16"), ("i8", "bf16"), ("i4", "f16"), ("f8", "bf16")])
@pytest.mark.parametrize("Nq,Hq,Hkv,D,L,causal", [
    (1, 8, 2, 128, 3000, False), (1, 64, 2, 64, 700, False), (16, 8, 2, 256, 1111, True), (128, 4, 4, 128, 900, True),
    (129, 4, 4, 128, 900, True), (2048, 8, 2, 128, 16384, True), (2048, 8, 1, 256, 2500, True), (1500, 14, 2, 64, 1700, True),
    (901, 10, 2, 128, 1000, True), (300, 128, 1, 128, 600, True), (77, 64, 1, 256, 513, False), (40, 8, 2, 96, 333, True)])
def test_weights_of_equal_terms_count_the_queries(Nq, Hq, Hkv, D, L, causal, kv, dtype):
    """Keys of zero and lse of zero: each term is exp(0) = 1, so an entry's weight is the number of (query, head)
    pairs that see it, exactly: no query vector, tile or limit may be lost or taken twice."""
    R = -(-L // 64) * 64
    g = synth.rng(390 + L)
    q = dev_bits(synth.normal_bits(g, (2, Nq, Hq, D), dtype), dtype)
    kd = {"i4": torch.zeros((R, Hkv, D // 2), dtype=torch.uint8), "i8": torch.zeros((R, Hkv, D), dtype=torch.int8),
          "f8": torch.zeros((R, Hkv, D), dtype=torch.uint8).view(torch.float8_e4m3fn)}.get(
              kv, torch.zeros((R, Hkv, D), dtype=q.dtype)).cuda()
    ks = torch.ones((R // 64, Hkv, 64), dtype=torch.float16, device="cuda") if kv in QUANT else None
    rows = torch.from_numpy(np.stack([g.permutation(R)[:L] for _ in range(2)]).astype(np.int32)).cuda()
    rows[0, L // 3] = -1
    lens = torch.tensor([L, L - L // 5], dtype=torch.int32, device="cuda")
    lse = torch.zeros((2, Nq, Hq), device="cuda")
    lse[1, Nq // 2] = -float("inf")                       # a query that saw nothing
    got = far.fa_rows_weights(q, kd, rows, 0.3, lse, kv_len=lens, causal=causal, k_scale=ks, check_status=True)
    j, i = torch.arange(L, device="cuda"), torch.arange(Nq, device="cuda")
    want = torch.zeros((2, L), device="cuda")
    for s, n in enumerate(lens.tolist()):
        see = ((rows[s] >= 0) & (j < n))[None].repeat(Nq, 1)
        if causal:
            see &= j[None] <= n - Nq + i[:, None]
        if s == 1:
            see &= (i != Nq // 2)[:, None]
        want[s] = see.sum(0) * (Hq // Hkv)
    assert torch.equal(got, want[:, None].expand(2, Hkv, L))
