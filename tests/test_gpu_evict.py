"""Eviction from row lists by accumulated weight (fa_kv_evict) against the oracle, entry for entry."""
import numpy as np
import pytest
import torch

import oracle
import synth
import row_indexed_flash_gb300 as far

pytestmark = pytest.mark.gpu


def make(seed, S, Hkv, L, lens=None, ties=False, pad=0.0, special=0.0):
    g = synth.rng(seed)
    acc = g.integers(0, 4, size=(S, Hkv, L)).astype(np.float32) if ties else np.exp(
        3 * g.standard_normal((S, Hkv, L))).astype(np.float32)
    rows = np.stack([g.permutation(4 * L)[:L] for _ in range(S)]).astype(np.int32)
    rows[g.random((S, L)) < pad] = -1
    if special:
        acc[g.random(acc.shape) < special] = np.nan
        acc[g.random(acc.shape) < special] = np.inf
        acc[g.random(acc.shape) < special] = -0.0
    return acc, rows, None if lens is None else np.asarray(lens, np.int32)


def check(acc, rows, lens, sinks, recent, k, extra=0, **kw):
    n = sinks + recent + k + extra
    want = oracle.evict(acc, rows, lens, sinks, recent, k, n)
    t = lambda a: None if a is None else torch.from_numpy(a).cuda()
    got = far.fa_kv_evict(t(acc), t(rows), t(lens), sinks, recent, k, out_len=n, **kw)
    for a, b, what in zip(got, want, ("rows", "len", "acc", "kept", "freed")):
        assert np.array_equal(a.cpu().numpy(), b, equal_nan=what == "acc"), what
    return got


@pytest.mark.parametrize("case", [
    dict(S=2, Hkv=2, L=1000, sinks=4, recent=64, k=188),
    dict(S=3, Hkv=3, L=77, sinks=2, recent=5, k=20, ties=True, pad=0.2),
    dict(S=1, Hkv=1, L=1, sinks=0, recent=0, k=1),
    dict(S=1, Hkv=8, L=1, sinks=0, recent=0, k=0),
    dict(S=4, Hkv=2, L=5000, lens=[0, 1, 4999, 2500], sinks=4, recent=16, k=300, ties=True),
    dict(S=2, Hkv=2, L=300, sinks=100, recent=300, k=10),                    # everything is kept
    dict(S=2, Hkv=2, L=300, lens=[12, 300], sinks=4, recent=8, k=5, extra=7),
    dict(S=2, Hkv=4, L=9001, sinks=0, recent=0, k=4500, ties=True, pad=0.5),
    dict(S=2, Hkv=4, L=4096, sinks=1, recent=1, k=0),
    dict(S=2, Hkv=4, L=20000, sinks=3, recent=7, k=19000, special=0.05, pad=0.01),
    dict(S=1, Hkv=16, L=70001, sinks=4, recent=508, k=8192, ties=True),
    dict(S=40, Hkv=2, L=3001, sinks=4, recent=100, k=400, pad=0.1),
])
def test_evict_matches_oracle(case):
    c = dict(case)
    sel = {x: c.pop(x, 0) for x in ("sinks", "recent", "k", "extra")}
    check(*make(500 + c["L"], **c), **sel)


def test_evict_of_only_padding_and_of_all_nan():
    acc, rows, _ = make(1, 2, 2, 500)
    rows[0] = -1
    acc[1] = np.nan
    check(acc, rows, None, 3, 5, 50)


def test_evict_beyond_what_shared_memory_holds():
    # 700,000 positions: more than the CTAs of a slice hold keys for
    acc, rows, _ = make(2, 1, 1, 700_000)
    total = torch.from_numpy(acc).cuda()
    got = far.fa_kv_evict(total, torch.from_numpy(rows).cuda(), None, 10, 100, 50_000)
    t = acc[0, 0]
    best = 10 + np.lexsort((np.arange(699_890), -t[10:-100]))[:50_000]
    keep = np.concatenate([np.arange(10), np.sort(best), np.arange(699_900, 700_000)])
    assert np.array_equal(got[3].cpu().numpy()[0], keep) and np.array_equal(got[0].cpu().numpy()[0], rows[0, keep])
    assert np.array_equal(got[2].cpu().numpy()[0, 0], t[keep])
    gone = np.setdiff1d(np.arange(700_000), keep)
    freed = got[4].cpu().numpy()[0]
    assert np.array_equal(freed[:len(gone)], rows[0, gone]) and (freed[len(gone):] == -1).all()


def test_evict_writes_the_callers_tensors_and_no_others():
    acc, rows, _ = make(3, 2, 2, 300)
    t = lambda a: torch.from_numpy(a).cuda()
    guard = [torch.full((s + 64,), 77, dtype=d, device="cuda") for s, d in
             ((2 * 40, torch.int32), (2, torch.int32), (2 * 2 * 40, torch.float32), (2 * 40, torch.int32), (2 * 300, torch.int32))]
    view = [g[:n].view(shape) for g, n, shape in zip(guard, (80, 2, 160, 80, 600), ((2, 40), (2,), (2, 2, 40), (2, 40), (2, 300)))]
    want = oracle.evict(acc, rows, None, 4, 6, 30, 40)
    far.fa_kv_evict(t(acc), t(rows), None, 4, 6, 30, out_len=40, rows_out=view[0], len_out=view[1], acc_out=view[2],
                    kept=view[3], freed=view[4])
    for v, w, g in zip(view, want, guard):
        assert np.array_equal(v.cpu().numpy(), w) and (g[-64:] == 77).all()


def test_evict_replays_in_a_graph():
    acc, rows, _ = make(4, 4, 2, 9000)
    a, r = torch.from_numpy(acc).cuda(), torch.from_numpy(rows).cuda()
    out = far.fa_kv_evict(a, r, None, 4, 100, 1000)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        far.fa_kv_evict(a, r, None, 4, 100, 1000, rows_out=out[0], len_out=out[1], acc_out=out[2], kept=out[3], freed=out[4])
    acc2, rows2, _ = make(5, 4, 2, 9000)
    a.copy_(torch.from_numpy(acc2))
    r.copy_(torch.from_numpy(rows2))
    graph.replay()
    for x, w in zip(out, oracle.evict(acc2, rows2, None, 4, 100, 1000, 1104)):
        assert np.array_equal(x.cpu().numpy(), w)


def test_decode_weights_evict_decode_as_a_serving_loop_does():
    # a cache over budget: attend, accumulate, evict, attend over what is left
    p = synth.random_problem(77, S=2, Nq=1, Hq=8, Hkv=2, D=128, R=4096, L=1500, pad_frac=0.0)
    dev = lambda a: torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda()
    q, k, v = dev(p.q), dev(p.k), dev(p.v)
    rows = torch.from_numpy(p.kv_rows).cuda()
    _, lse = far.fa_rows_decode(q, k, v, rows, p.scale, want_lse=True)
    acc = far.fa_rows_weights(q, k, rows, p.scale, lse)
    new_rows, n, new_acc, kept, freed = far.fa_kv_evict(acc, rows, None, 4, 60, 448, out_len=600)
    assert n.tolist() == [512, 512] and (freed >= 0).sum(dim=1).tolist() == [988, 988]
    want = oracle.evict(acc.cpu().numpy(), p.kv_rows, None, 4, 60, 448, 600)
    assert np.array_equal(kept.cpu().numpy(), want[3])
    out, lse2 = far.fa_rows_decode(q, k, v, new_rows, p.scale, kv_len=n, want_lse=True)
    ref, ref_lse = oracle.attend_rows(oracle.widen_bf16(p.q), p.k, p.v, new_rows.cpu().numpy(), p.scale, kv_format="bf16",
                                      kv_len=n.cpu().numpy())
    assert np.abs(out.cpu().numpy() - ref).max() <= 2e-3
    # the totals that went on with the list still line up with it
    again = far.fa_rows_weights(q, k, new_rows, p.scale, lse2, new_acc, kv_len=n)
    assert again is new_acc and (again[:, :, 512:] == 0).all()
    both = set(new_rows[0, :512].tolist()) | set(freed[0, :988].tolist())
    assert both == set(p.kv_rows[0].tolist())
