"""Calls given a stream other than the current one: what they allocate belongs to that stream."""
import numpy as np
import pytest
import torch

import synth
import row_indexed_flash_gb300 as far

from helpers import dev_bits

pytestmark = pytest.mark.gpu

BUSY = 200_000_000      # clocks, about 0.1 s


def problem():
    p = synth.random_problem(700, S=2, Nq=1, Hq=8, Hkv=2, D=128, R=4096, L=2000, pad_frac=0.0)
    q, k, v = (dev_bits(x, "bf16") for x in (p.q, p.k, p.v))
    return q, k, v, torch.from_numpy(p.kv_rows).cuda(), p.scale


def junk(*shapes):
    """Freed blocks of these sizes that hold anything but zeros."""
    torch.cuda.synchronize()
    for t in [torch.full(s, 7, dtype=torch.int32, device="cuda") for s in shapes for _ in range(3)]:
        del t
    torch.cuda.synchronize()


@pytest.mark.parametrize("as_handle", [False, True])
def test_new_accumulator_is_zeroed_before_the_kernel(as_handle):
    q, k, v, rows, scale = problem()
    _, lse = far.fa_rows_decode(q, k, v, rows, scale, want_lse=True)
    want = far.fa_rows_weights(q, k, rows, scale, lse)
    other = torch.cuda.Stream()
    junk((2, 2, 2000))
    torch.cuda._sleep(BUSY)                             # the current stream does nothing for a while
    got = far.fa_rows_weights(q, k, rows, scale, lse, stream=other.cuda_stream if as_handle else other)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_default_stream_by_its_handle():
    q, k, v, rows, scale = problem()
    _, lse = far.fa_rows_decode(q, k, v, rows, scale, want_lse=True)
    want = far.fa_rows_weights(q, k, rows, scale, lse)
    assert torch.equal(far.fa_rows_weights(q, k, rows, scale, lse, stream=torch.cuda.default_stream().cuda_stream), want)


def test_status_is_read_on_the_call_s_stream():
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    junk((1,))
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        torch.cuda._sleep(BUSY)
        ws.view(torch.int32)[0] = far.FA_WS_WAIT_EXPIRED
    assert far.fa_rows_status(ws, clear=True, stream=other) == far.FA_WS_WAIT_EXPIRED
    assert far.fa_rows_status(ws, stream=other) == 0


def test_outputs_do_not_take_memory_that_the_current_stream_still_reads():
    q, k, v, rows, scale = problem()
    acc = torch.rand((2, 2, 2000), device="cuda")
    table = torch.arange(64, dtype=torch.int32, device="cuda")[None].repeat(2, 1)
    lens = torch.full((2,), 4096, dtype=torch.int32, device="cuda")
    lo, hi = (torch.zeros((64, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    score, first = torch.rand((2, 2, 64), device="cuda"), acc[:, 0].contiguous()
    head_rows = rows[:, None].repeat(1, 2, 1)
    x = dev_bits(synth.normal_bits(synth.rng(701), (4096, 2, 128), "bf16"), "bf16")
    other = torch.cuda.Stream()
    calls = [
        lambda s: far.fa_rows_decode(q, k, v, rows, scale, want_lse=True, stream=s),
        lambda s: far.fa_rows_prefill(q, k, v, rows, scale, want_lse=True, stream=s),
        lambda s: far.fa_rows_decode_heads(q, k, v, head_rows, scale, want_lse=True, stream=s),
        lambda s: far.fa_kv_evict(acc, rows, None, 1, 1, 498, stream=s),
        lambda s: (far.fa_kv_block_scores(q, lo, hi, table, lens, stream=s),),
        lambda s: far.fa_kv_block_rows(score, table, lens, 1, 1, 6, stream=s),
        lambda s: (far.fa_kv_page_table_to_rows(table, lens, 4096, stream=s),),
        lambda s: far.fa_kv_quantize_int8(x, 4096, stream=s),
        lambda s: (far.fa_kv_sparse_rows(first, 4, 8, 100, stream=s),),
    ]
    for i, call in enumerate(calls):
        outs = call(None)                              # warm, and the sizes of what the call allocates
        sizes = [t.numel() * t.element_size() for t in outs if t is not None]
        torch.cuda.synchronize()
        mine = [torch.full((n,), 3, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        copies = [t.clone() for t in mine]             # still to be read ...
        del mine                                       # ... when the blocks are free for the current stream
        got = call(other)
        torch.cuda.synchronize()
        assert all((c == 3).all() for c in copies), i
        for a, b in zip(got, outs):
            assert a is None and b is None or torch.equal(a, b), i
