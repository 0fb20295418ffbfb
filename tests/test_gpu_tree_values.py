"""Attention of drafted trees (fa_rows_tree) over values that are not finite, where calls have many short units of work."""
import pytest
import torch

import synth
from branch_helpers import kin_of
from test_gpu_tree import Problem

pytestmark = pytest.mark.gpu


def same_but_nan(got, want):
    """Equal bits, NaN exactly where it is wanted."""
    return torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("kv,q", [("f8", "bf16"), ("f8", "f16"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("S,T,Hq,lo,hi", [(150, 6, 16, 20, 64), (150, 6, 16, 20, 128), (150, 40, 32, 40, 64), (150, 40, 32, 40, 128),
                                          (400, 3, 8, 3, 40)])
@pytest.mark.parametrize("layout", ["runs", "shuffled"])
def test_a_nan_in_one_nodes_v_reaches_exactly_those_that_see_it(kv, q, S, T, Hq, lo, hi, layout):
    """Lists of one or two tiles, so that every CTA goes through many (slice, KV head) pairs while loads and conversions run
    ahead.  K stays as it is: weights and all other components keep their bits."""
    Hkv, D = 8, 128
    g = synth.rng(S + T + hi)
    lens = g.integers(lo, hi + 1, S).tolist()
    p = Problem(50 + T, kv=kv, q=q, S=S, T=T, Hq=Hq, Hkv=Hkv, D=D, L=hi, lens=lens, layout=layout)
    want, want_lse = p.call()
    kin = kin_of(p.parent.cpu().numpy())
    v = p.v.view(torch.uint8) if kv == "f8" else p.v
    G = Hq // Hkv
    for s in range(S):
        u, c = s % T, 37 * s % D
        row = int(p.rows[s, lens[s] - T + u])
        for h in {s % Hkv, 5 * s % Hkv}:
            v[row, h, c] = 0x7f if kv == "f8" else float("nan")     # 0x7f: the NaN of E4M3
            for t in range(T):
                if kin[s, t, u]:
                    want[s, t, h * G:(h + 1) * G, c] = float("nan")
    for _ in range(4):
        out, lse = p.call(check_status=True)
        assert torch.equal(lse, want_lse)
        assert same_but_nan(out, want)
