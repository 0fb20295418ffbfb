"""Calls captured into graphs without a workspace of the caller's: each graph stands for itself."""
import pytest
import torch

import synth
import row_indexed_flash_gb300 as far

from helpers import dev_bits

pytestmark = pytest.mark.gpu


def attention(seed, kind, S, L):
    p = synth.random_problem(seed, S=S, Nq=100 if kind.startswith("prefill") else 1, Hq=8, Hkv=2, D=128, R=8192, L=L,
                             pad_frac=0.0)
    q, k, v = (dev_bits(x, "bf16") for x in (p.q, p.k, p.v))
    rows = torch.from_numpy(p.kv_rows).cuda()
    kw = dict(want_lse=True)
    if kind == "decode_i8":
        (k, kw["k_scale"]), (v, kw["v_scale"]) = (far.fa_kv_quantize_int8(x, p.R) for x in (k, v))
    if kind.endswith("heads"):
        rows = rows[:, None].repeat(1, 2, 1)
    if kind.startswith("prefill") and seed % 2:
        rows = (rows // 128)[..., :1] * 128 + torch.arange(rows.shape[-1], device="cuda", dtype=torch.int32)   # one run:
        rows = rows.clamp(max=8191).int()                                                                       # another mode
    fn = getattr(far, {"decode": "fa_rows_decode", "decode_i8": "fa_rows_decode", "decode_heads": "fa_rows_decode_heads",
                       "prefill": "fa_rows_prefill", "prefill_heads": "fa_rows_prefill_heads"}[kind])
    return lambda: fn(q, k, v, rows, p.scale, **kw)


@pytest.mark.parametrize("kind", ["decode", "decode_i8", "decode_heads", "prefill", "prefill_heads"])
def test_graphs_share_no_scratch(kind):
    calls = [attention(1000, kind, 1, 8000), attention(1001, kind, 2, 6000)]
    want = [[t.clone() for t in c()] for c in calls]
    stream = torch.cuda.Stream()
    graphs, outs = [], []
    stream.wait_stream(torch.cuda.current_stream())
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            outs.append(c())
        graphs.append(g)
    # what the binding keeps for that stream belongs to no graph
    assert far.default_workspace(stream=stream, is_prefill=kind.startswith("prefill")) is None
    # the second one alone, first of all: nothing relies on a replay of the other
    for i in (1, 0):
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i])), i
    sides = [torch.cuda.Stream() for _ in graphs]
    for t in (x for o in outs for x in o):
        t.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(40):
        for g, s in zip(graphs, sides):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i])), i


def test_weights_and_scores_captured_first_leave_nothing_behind():
    p = synth.random_problem(1010, S=2, Nq=1, Hq=8, Hkv=2, D=128, R=512, L=300)
    q, k = dev_bits(p.q, "bf16"), dev_bits(p.k, "bf16")
    rows, lse = torch.from_numpy(p.kv_rows).cuda(), torch.zeros((2, 1, 8), device="cuda")
    lo, hi = (torch.ones((8, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, n = torch.arange(8, dtype=torch.int32, device="cuda")[None].repeat(2, 1), torch.full((2,), 500, dtype=torch.int32, device="cuda")
    want = far.fa_rows_weights(q, k, rows, p.scale, lse), far.fa_kv_block_scores(q, lo, hi, table, n)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        got = far.fa_rows_weights(q, k, rows, p.scale, lse), far.fa_kv_block_scores(q, lo, hi, table, n)
    assert far.default_workspace(stream=stream, is_prefill=True) is None
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(stream):
        assert torch.equal(far.fa_rows_weights(q, k, rows, p.scale, lse, check_status=True), want[0])
