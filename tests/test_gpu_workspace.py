"""Calls of different shapes that use one decode workspace in turn: neither sees what the other left there."""
import numpy as np
import pytest
import torch

import synth
import row_indexed_flash_gb300 as far

from helpers import dev_bits

pytestmark = pytest.mark.gpu


def call(kind, seed, S, Hkv, L, G=4, Nq=1, heads=False):
    """A decode into an output of NaN: call(workspace) -> (out, lse); its workspace bytes."""
    D = 64 if kind == "bf16_d64" else 128
    p = synth.random_problem(seed, S=S, Nq=Nq, Hq=G * Hkv, Hkv=Hkv, D=D, R=8192, L=L, pad_frac=0.0)
    q, k, v = (dev_bits(x, "bf16") for x in (p.q, p.k, p.v))
    kw = {}
    if kind in ("i8", "f8", "i4"):
        quant = {"i8": far.fa_kv_quantize_int8, "f8": far.fa_kv_quantize_fp8, "i4": far.fa_kv_quantize_int4}[kind]
        (k, ks), (v, vs) = quant(k, p.R), quant(v, p.R)
        kw = dict(k_scale=ks, v_scale=vs)
    rows = torch.from_numpy(p.kv_rows).cuda()
    a, _, _ = far.make_args(q, k, v, rows, p.scale, **kw)
    need = far.fa_rows_workspace_size(a)
    fn = far.fa_rows_decode
    if heads:
        rows, fn = rows[:, None].repeat(1, Hkv, 1), far.fa_rows_decode_heads

    def run(ws):
        out = torch.full((S, Nq, G * Hkv, D), float("nan"), device="cuda")
        lse = torch.full((S, Nq, G * Hkv), float("nan"), device="cuda")
        return fn(q, k, v, rows, p.scale, out=out, lse=lse, workspace=ws, **kw)
    return run, need


@pytest.mark.parametrize("heads", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "i8", "f8", "i4", "bf16_d64"])
def test_calls_of_any_shapes_share_a_workspace(kind, heads):
    # few (slice, KV head) pairs with many splits, then more pairs than the first one had counters for
    calls = [call(kind, 900, 1, 2, 8000, heads=heads), call(kind, 901, 23, 8, 1984, heads=heads), call(kind, 902, 3, 1, 6000, heads=heads),
             call(kind, 903, 2, 40, 3000, G=1, heads=heads), call(kind, 904, 1, 1, 64, heads=heads)]
    assert sum(n > 16384 for _, n in calls) >= 3                    # those have splits
    size = max(n for _, n in calls)
    want = [run(torch.zeros(n, dtype=torch.uint8, device="cuda")) for run, n in calls]
    assert all(torch.isfinite(t).all() for w in want for t in w)
    one = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for i in (0, 1, 2, 1, 3, 0, 4, 3, 2, 1, 1):
        for a, b in zip(calls[i][0](one), want[i]):
            assert torch.equal(a, b), i
    # the binding's own workspace, which grows
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for i in (4, 0, 1, 2, 3, 1):
            got = calls[i][0](None)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want[i])), i


def test_more_pairs_than_the_fixed_counters():
    run, need = call("bf16_d64", 905, 4100, 1, 4096, G=2)           # at most 2,048 entries a CTA there
    assert need > 4100 * 2 * 2 * 64 * 4                             # two splits at least
    few, few_need = call("bf16", 906, 2, 1, 8000)
    out, lse = run(torch.zeros(need, dtype=torch.uint8, device="cuda"))
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    first = few(ws)
    ws[16384:] = 0x5A                                               # what any partials may leave
    for _ in range(2):
        a, b = run(ws)
        assert torch.equal(a, out) and torch.equal(b, lse)
    again = few(ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
