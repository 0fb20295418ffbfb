"""Host-side refusals of the cache-reduction entry points: a status and a text, nothing launched (CPU)."""
import ctypes

import pytest
import torch

import row_indexed_flash_gb300 as far

from test_abi import _args, lib  # noqa: F401

P = 4096        # a pointer that no accepted call would be given


def weights(lib, lse=P, decay=1.0, acc=P, ws=P, ws_bytes=256, **kw):
    return lib.fa_rows_weights(ctypes.byref(_args(**kw)), lse, decay, acc, ws, ws_bytes, None)


def test_weights_refusals(lib):
    assert lib.fa_rows_weights(None, P, 1.0, P, P, 256, None) == 1
    assert weights(lib, lse=None) == 1 and weights(lib, lse=P + 2) == 1
    assert weights(lib, acc=None) == 1 and weights(lib, acc=P + 1) == 1
    assert weights(lib, decay=float("nan")) == 1 and weights(lib, decay=float("inf")) == 1
    assert weights(lib, ws=None) == 3 and weights(lib, ws_bytes=255) == 3
    assert weights(lib, Hq=6, Hkv=4) == 1 and weights(lib, k=P + 8) == 1
    assert weights(lib, kv_dtype=far.FA_I8) == 1                                # no scales
    assert weights(lib, D=260) == 2 and weights(lib, D=100) == 2 and weights(lib, S=70000) == 2
    assert weights(lib, mask_kind=far.FA_MASK_DENSE) == 1
    assert weights(lib, S=0) == 0 and weights(lib, Nq=0) == 0 and weights(lib, list_len=0) == 0
    assert weights(lib, S=-1) == 1 and far.fa_last_error()


def test_head_list_refusals(lib):
    for fn in (lib.fa_rows_decode_heads, lib.fa_rows_prefill_heads):
        assert fn(None, P, 256, None) == 1
        a = _args(mask_kind=far.FA_MASK_DENSE, mask=P)
        assert fn(ctypes.byref(a), P, 256, None) == 2 and "per KV head" in far.fa_last_error()
        assert fn(ctypes.byref(_args(S=1 << 16, Hkv=1 << 15, Hq=1 << 15)), P, 256, None) == 2
        assert fn(ctypes.byref(_args(Hq=6, Hkv=4)), P, 256, None) == 1


def evict(lib, acc=1 << 20, rows=2 << 20, lens=3 << 20, S=2, Hkv=2, L=64, sinks=1, recent=1, k=2, acc_out=4 << 20,
          rows_out=5 << 20, len_out=6 << 20, out_len=4, kept=7 << 20, freed=8 << 20):
    return lib.fa_kv_evict(acc, rows, lens, S, Hkv, L, sinks, recent, k, acc_out, rows_out, len_out, out_len, kept, freed, None)


def test_evict_refusals(lib):
    assert evict(lib, out_len=3) == 1 and evict(lib, k=-1) == 1 and evict(lib, Hkv=0) == 1
    assert evict(lib, acc=None) == 1 and evict(lib, rows=None) == 1 and evict(lib, len_out=None) == 1
    assert evict(lib, acc_out=None) == 1 and evict(lib, rows_out=None) == 1 and evict(lib, acc=(1 << 20) + 2) == 1
    assert evict(lib, rows_out=2 << 20) == 1 and "overlaps" in far.fa_last_error()
    assert evict(lib, acc_out=(1 << 20) + 4 * 255) == 1                         # the last total
    assert evict(lib, kept=(5 << 20) + 4) == 1 and "overlap" in far.fa_last_error()
    assert evict(lib, S=70000) == 2 and evict(lib, L=(1 << 30) + 1) == 2
    assert evict(lib, S=0) == 0


def test_block_refusals(lib):
    def bounds(k=P, dt=far.FA_BF16, ks=None, R=128, Hkv=2, D=128, pages=P, fill=P, n=2, lo=P, hi=P, bt=far.FA_BF16):
        return lib.fa_kv_block_bounds(k, dt, ks, R, Hkv, D, pages, fill, n, lo, hi, bt, None)
    assert bounds(R=100) == 2 and bounds(D=100) == 2 and bounds(D=512) == 2 and bounds(dt=far.FA_F32) == 2
    assert bounds(bt=far.FA_F16) == 2 and bounds(bt=far.FA_F32, dt=far.FA_I8, ks=P) == 2
    assert bounds(dt=far.FA_I8) == 1 and bounds(k=P + 8) == 1 and bounds(pages=None) == 1 and bounds(n=-1) == 1
    assert bounds(n=0) == 0

    def scores(q=P, dt=far.FA_BF16, S=2, Nq=1, Hq=8, Hkv=2, D=128, n_seq=2, NB=4, table=P, lens=P, seq=None, out=P, ws=P, wb=256):
        return lib.fa_kv_block_scores(q, dt, S, Nq, Hq, Hkv, D, P, P, 100, table, n_seq, NB, lens, seq, out, ws, wb, None)
    assert scores(D=96) == 2 and scores(dt=far.FA_F32) == 2 and scores(Hq=6, Hkv=4) == 1 and scores(q=P + 2) == 1
    assert scores(n_seq=1) == 1 and scores(table=None) == 1 and scores(out=None) == 1 and scores(ws=None) == 3
    assert scores(wb=100) == 3 and scores(NB=1 << 26) == 1 and scores(S=70000, n_seq=70000) == 2
    assert scores(S=0) == 0 and scores(Nq=0) == 0

    def rows(score=P, table=P, n_seq=2, NB=4, lens=P, seq=None, S=2, Hkv=2, a=1, b=1, k=2, out=P, ln=P, L=256):
        return lib.fa_kv_block_rows(score, table, n_seq, NB, lens, seq, S, Hkv, a, b, k, out, ln, L, None)
    assert rows(L=255) == 1 and rows(k=-1) == 1 and rows(n_seq=1) == 1 and rows(score=None) == 1 and rows(ln=None) == 1
    assert rows(out=None) == 1 and rows(NB=1 << 26) == 1 and rows(S=70000, n_seq=70000) == 2 and rows(S=0) == 0


def test_binding_checks_shapes_before_pointers():
    q = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16)
    k = torch.zeros((64, 2, 64), dtype=torch.bfloat16)
    rows = torch.zeros((1, 8), dtype=torch.int32)
    lse = torch.zeros((1, 1, 4))
    for bad in (dict(lse=lse[..., :2]), dict(kv_rows=rows.long()), dict(acc=torch.zeros((1, 2, 7))),
                dict(kv_len=torch.zeros(2, dtype=torch.int32)), dict(mask=torch.zeros((1, 2, 8)))):
        kw = dict(kv_rows=rows, scale=1.0, lse=lse)
        kw.update(bad)
        with pytest.raises(ValueError):
            far.fa_rows_weights(q, k, **kw)
    with pytest.raises(ValueError):                       # one list per slice where one per head is wanted
        far.fa_rows_decode_heads(q, k, k, rows, 1.0)
    with pytest.raises(ValueError):
        far.fa_kv_evict(torch.zeros((1, 2, 8)), torch.zeros((1, 7), dtype=torch.int32), None, 1, 1, 1)
    with pytest.raises(ValueError):
        far.fa_kv_block_bounds(k, rows[0], None, torch.zeros((1, 2, 64), dtype=torch.bfloat16), torch.zeros((1, 2, 32)))
    with pytest.raises(ValueError):
        far.fa_kv_block_scores(q, torch.zeros((1, 2, 64)), torch.zeros((1, 2, 64)), rows, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        far.fa_kv_block_rows(torch.zeros((1, 2, 9)), rows, torch.zeros(1, dtype=torch.int32), 1, 1, 1)


def test_binding_refuses_scales_of_another_pool():
    q = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16)
    k = torch.zeros((128, 2, 64), dtype=torch.int8)
    rows = torch.zeros((1, 8), dtype=torch.int32)
    bound = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    for ks in (None, torch.zeros((1, 2, 64), dtype=torch.float16), torch.zeros((2, 2, 64))):
        with pytest.raises(ValueError, match="k_scale"):
            far.fa_rows_weights(q, k, rows, 1.0, torch.zeros((1, 1, 4)), k_scale=ks)
        with pytest.raises(ValueError, match="k_scale"):
            far.fa_kv_block_bounds(k, rows[0], None, bound, bound.clone(), k_scale=ks)


@pytest.mark.parametrize("ks", [
    torch.zeros((2, 2, 64), dtype=torch.bfloat16), torch.zeros((2, 2, 64), dtype=torch.int16),
    torch.zeros((128, 2), dtype=torch.float16), torch.zeros((2, 64, 2), dtype=torch.float16),
    torch.zeros((1, 4, 64), dtype=torch.float16), torch.zeros(256, dtype=torch.float16)])
def test_binding_refuses_scales_of_another_type_or_layout(ks):
    q = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16)
    rows = torch.zeros((1, 8), dtype=torch.int32)
    bound = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    for k in (torch.zeros((128, 2, 64), dtype=torch.int8), torch.zeros((128, 2, 32), dtype=torch.uint8),
              torch.zeros((128, 2, 64), dtype=torch.float8_e4m3fn)):
        with pytest.raises(ValueError, match="k_scale"):
            far.fa_rows_weights(q, k, rows, 1.0, torch.zeros((1, 1, 4)), k_scale=ks)
        with pytest.raises(ValueError, match="k_scale"):
            far.fa_kv_block_bounds(k, rows[0], None, bound, bound.clone(), k_scale=ks)
        fine = torch.zeros((2, 2, 64), dtype=torch.float16)
        for kw in (dict(k_scale=ks, v_scale=fine), dict(k_scale=fine, v_scale=ks)):
            with pytest.raises(ValueError, match="float16"):
                far.fa_rows_decode_heads(q, k, k, rows[None], 1.0, **kw)


def test_binding_finds_the_current_stream_by_the_public_interface_too(monkeypatch):
    class Stream:
        cuda_stream = 4711
    asked = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: asked.append(device) or Stream())
    monkeypatch.setattr(far, "_raw_stream", None)      # a torch without the private function
    for device in (torch.device("cuda", 1), torch.device("cuda")):
        assert far._stream(None, device) == 4711
    assert asked == [torch.device("cuda", 1), torch.device("cuda")]
    monkeypatch.setattr(far, "_raw_stream", lambda index: 100 + index)
    assert far._stream(None, torch.device("cuda", 1)) == 101 and far._stream(None, torch.device("cuda")) == 4711
    assert far._stream(Stream(), torch.device("cuda", 1)) == 4711 and far._stream(12, torch.device("cuda", 1)) == 12


def test_binding_takes_scales_of_the_pool():
    # past the shape checks: refused for being on the host
    k, ks = torch.zeros((128, 2, 64), dtype=torch.int8), torch.zeros((2, 2, 64), dtype=torch.float16)
    bound = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        far.fa_kv_block_bounds(k, torch.zeros(1, dtype=torch.int32), None, bound, bound.clone(), k_scale=ks)
