"""Quantised decode where the values cancel: keys seen alike, codes of either sign, so that an output is far
smaller than the values it averages.

With q = 0 every logit is 0 and the output is the mean of the listed values.  Its error is bounded by the mean
magnitude a = sum p |v| times
  2^-12            each O weight is one f16 value,
  2^-14            the tensor core's sums, each cut off by at most 2^-23 of the running sum: at most 12,000 / 16
                   steps of an f16 product in one chain, 750 * 2^-23 < 2^-13.4 in the worst case of one sign, and
                   half of that on average over a chain that grows evenly.
"""
import numpy as np
import pytest
import torch

import synth
import row_indexed_flash_gb300 as far

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [False, True])
@pytest.mark.parametrize("kv", ["i8", "i4", "f8"])
@pytest.mark.parametrize("S,Nq,Hq,Hkv,L", [(1, 1, 2, 2, 12000), (15, 1, 8, 8, 3008), (2, 1, 8, 2, 1216), (1, 1, 32, 4, 9000),
                                         (1, 2, 8, 1, 12000), (1, 4, 32, 4, 5000), (64, 1, 8, 8, 700)])
def test_outputs_of_values_that_cancel(kv, S, Nq, Hq, Hkv, L, heads):
    D, R = 128, 16384
    g = synth.rng(920 + L + S)
    if kv == "i8":
        codes = np.clip(np.rint(g.standard_normal((R, Hkv, D)) * 40), -127, 127).astype(np.int8)
        vd, values = torch.from_numpy(codes).cuda(), codes.astype(np.float64)
    elif kv == "i4":
        codes = np.clip(np.rint(g.standard_normal((R, Hkv, D)) * 3), -7, 7).astype(np.int64)
        packed = ((codes[..., 0::2] & 15) | ((codes[..., 1::2] & 15) << 4)).astype(np.uint8)
        vd, values = torch.from_numpy(packed).cuda(), codes.astype(np.float64)
    else:
        x = np.clip(g.standard_normal((R, Hkv, D)) * 100, -448, 448)   # E4M3 holds no more
        vd = torch.from_numpy(x.astype(np.float32)).cuda().to(torch.float8_e4m3fn)
        values = vd.float().double().cpu().numpy()
    scale = torch.from_numpy((g.random((R // 64, Hkv, 64)) * 0.01 + 0.01).astype(np.float16)).cuda()
    s = scale.cpu().numpy().astype(np.float64).transpose(0, 2, 1).reshape(R, Hkv)
    values = values * s[..., None]
    rows = np.stack([g.permutation(R)[:L] for _ in range(S)]).astype(np.int32)
    q = torch.zeros((S, Nq, Hq, D), dtype=torch.bfloat16, device="cuda")
    rd, fn = torch.from_numpy(rows).cuda(), far.fa_rows_decode
    if heads:
        rd, fn = rd[:, None].repeat(1, Hkv, 1), far.fa_rows_decode_heads
    for hint in (0, S * L):
        out, _ = fn(q, vd, vd, rd, 0.1, k_scale=scale, v_scale=scale, n_valid_hint=hint, check_status=True)
        out = out.double().cpu().numpy()
        for i in range(S):
            v = values[rows[i]]                                              # [L, Hkv, D]
            want = np.repeat(v.mean(axis=0), Hq // Hkv, axis=0)
            size = np.repeat(np.abs(v).mean(axis=0), Hq // Hkv, axis=0)
            err = np.abs(out[i] - want[None]) / size[None]
            assert err.max() <= 2.0 ** -12 + 2.0 ** -14, (i, err.max())


@pytest.mark.parametrize("heads", [False, True])
@pytest.mark.parametrize("qtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,S,Nq,Hq,Hkv,L", [(256, 1, 1, 2, 2, 3008), (256, 2, 1, 8, 2, 700), (256, 40, 2, 8, 8, 1000),
                                          (256, 1, 1, 8, 1, 64), (128, 2, 1, 8, 2, 3008), (64, 2, 1, 8, 2, 3008)])
@pytest.mark.parametrize("depth", [2.0, 5.0, 9.0])
def test_int8_outputs_of_small_weights(depth, D, S, Nq, Hq, Hkv, L, qtype, heads):
    """One entry with logit 0, the others with -depth, and every value v = 1 code times its scale: the output is v
    times the sum of the rounded P over the sum of P.

    P is carried to 16 bits (2^-17) or is one f16 weight of its own reference (2^-12, the quantised kernel at D 128);
    the tensor core's sums take at most 8 steps per tile of 64 keys, 376 in all, each cut off by at most 2^-23, and
    the row sums some 2^-23: 2^-14 and 2^-11.5 bound them.
    """
    R = 4096
    g = synth.rng(930)
    rows = np.stack([g.permutation(R)[:L] for _ in range(S)]).astype(np.int32)
    rows[:, 0] = 0
    rows[:, 1:][rows[:, 1:] == 0] = 1
    k = torch.zeros((R, Hkv, D), dtype=torch.int8, device="cuda")
    k[1:, :, 0] = -1
    v = torch.ones((R, Hkv, D), dtype=torch.int8, device="cuda")
    ones = torch.ones((R // 64, Hkv, 64), dtype=torch.float16, device="cuda")
    q = torch.zeros((S, Nq, Hq, D), dtype=qtype, device="cuda")
    q[..., 0] = 1.0
    rd, fn = torch.from_numpy(rows).cuda(), far.fa_rows_decode
    if heads:
        rd, fn = rd[:, None].repeat(1, Hkv, 1), far.fa_rows_decode_heads
    for scale in (0.0241, 0.9, 500.0):
        vs = ones * scale
        out, _ = fn(q, k, v, rd, depth, k_scale=ones, v_scale=vs, check_status=True)
        err = (out.double() / vs[0, 0, 0].double() - 1).abs().max().item()
        assert err <= (2.0 ** -11.5 if D == 128 else 2.0 ** -14), (scale, err)
