"""Attention of drafted trees (fa_rows_tree): values that are not finite, many short lists, the precision of weights."""
import pytest
import torch

import synth
from branch_helpers import assert_near, kin_of
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


@pytest.mark.parametrize("kv,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f16", 64), ("f16", 128), ("f16", 256),
                                  ("bf16", 96), ("f16", 40)])
@pytest.mark.parametrize("T,Hq,L,spread", [(5, 8, 150, 1.0), (40, 32, 700, 1.0), (12, 8, 9000, 1.0), (5, 8, 190, 12.0)])
def test_infinities_of_the_context_come_out_as_infinities(kv, D, T, Hq, L, spread):
    """Every node sees them with a weight above 0: an infinity where all of a component have one sign, else NaN.  spread: the
    weights go down to e^-80 of the largest, far below the 16-bit types of the product."""
    p = Problem(60, kv=kv, q=kv, S=2, T=T, Hq=Hq, Hkv=2, D=D, L=L, layout="pages", nodes=[T, T - 2], amp=spread,
                scale=0.3 * D ** -0.5 * 3)
    want, want_lse = p.call()
    G, inf, nan = Hq // 2, float("inf"), float("nan")
    for s, live in ((0, T), (1, T - 2)):
        for entries, h, c, x, to in (([0], 0, 5, [inf], inf), ([L // 2], 1, 7, [-inf], -inf), ([3, 70], 0, D - 1, [inf, -inf], nan),
                                     ([L - T - 1], 1, 16, [nan], nan), ([9, 80, 90], 1, 17, [-inf] * 3, -inf)):
            for e, y in zip(entries, x):
                p.v[int(p.rows[s, e]), h, c] = y
            want[s, :live, h * G:(h + 1) * G, c] = to
    out, lse = p.call()
    assert torch.equal(lse, want_lse) and same_but_nan(out, want)


def test_every_value_of_a_long_context_infinite():
    p = Problem(61, S=1, T=4, L=100000, layout="pages", Hq=2, Hkv=1)
    p.v[:, 0, ::2] = float("inf")
    p.v[:, 0, 1::2] = float("-inf")
    p.v[p.rows[0, -4:].long()] = 1.0                       # the nodes' own are finite
    out, _ = p.call(check_status=True)
    assert (out[..., ::2] == float("inf")).all() and (out[..., 1::2] == float("-inf")).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,Hq,L", [(4, 4, 12), (7, 8, 40), (40, 32, 64)])
def test_weights_over_f16_pools_keep_more_than_one_f16_value(D, T, Hq, L):
    """Logits near one another, so that a logit's own error is small: with weights of one f16 value (off by up to 2^-12) the
    outputs miss the bound, as a pair of f16 (off by up to 2^-22, or 2^-32 of the largest) they hold it."""
    p = Problem(70, kv="f16", q="f16", S=3, T=T, Hq=Hq, Hkv=2, D=D, L=L, amp=0.05)
    assert_near(*p.call(), p.want(), D, 20, T, 1.0)
