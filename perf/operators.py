"""Cases for timing the cache-reduction operators of the row-indexed attention library.

Two ways to spend less on a long KV cache, each with the calls a serving loop makes of it:

* eviction by accumulated attention weight: ``weights`` adds the softmax weight every listed cache
  entry received to a running total, ``evict`` keeps the sinks, the recent entries and the heaviest
  of the rest, and compacts the row list and the totals;
* attention over selected 64-row blocks: ``bounds`` keeps the elementwise minimum and maximum of
  each page's keys, ``scores`` bounds the logit any key of a block can reach, ``block_rows`` turns
  the best blocks of every (slice, KV head) into row lists, and ``heads`` attends over lists of that
  kind.

``run`` computes them with elementary torch operations in 32 bits (``own`` false) or through the
library's entry points (``own`` true).
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # one new token of each of four sequences of a shuffled 65,536-row pool: the weights its
        # attention step gave, added to the totals
        dict(name="weights_token_bf16", op="weights", kv="bf16", q="bf16", S=4, Nq=1, Hq=32, Hkv=8, D=128, n=16384,
             ragged=False, layout="shuffled", causal=False),
        # a 2,048-token prompt chunk at the end of 16,384 tokens written in long runs
        dict(name="weights_prompt_bf16", op="weights", kv="bf16", q="bf16", S=1, Nq=2048, Hq=32, Hkv=8, D=128,
             n=16384, ragged=False, layout="runs", causal=True),
        # two short sequences over budget: the smallest call, where latency counts
        dict(name="evict_small", op="evict", S=2, Hkv=2, n=1000, L=1024, ragged=False, sinks=4, recent=64, k=188),
        # four 99,936-token prompts cut to 16,384 entries each
        dict(name="evict_prompts", op="evict", S=4, Hkv=8, n=99936, L=99936, ragged=False, sinks=4, recent=508,
             k=15872),
        # after a token of each of 32 sequences: the pages they were appended to
        dict(name="bounds_token_bf16", op="bounds", kv="bf16", q="bf16", Hkv=8, D=128, pages=32, pool_pages=2048,
             full=False),
        # after a 99,936-token prompt into an INT8 pool of 400,000 rows
        dict(name="bounds_prompt_i8", op="bounds", kv="i8", q="bf16", Hkv=8, D=128, pages=1562, pool_pages=6250,
             full=True),
        # a token of each of 32 sequences of 1k to 128k tokens
        dict(name="scores_token_bf16", op="scores", q="bf16", S=32, Nq=1, Hq=32, Hkv=8, D=128, n=131072, lo=1024,
             one_seq=False),
        # a 2,048-token prompt chunk in tiles of 128 queries, at the end of 99,936 tokens
        dict(name="scores_prompt_bf16", op="scores", q="bf16", S=16, Nq=128, Hq=32, Hkv=8, D=128, n=99936, lo=0,
             one_seq=True),
        # the best 29 blocks of each (sequence, KV head), the first one and the last two
        dict(name="block_rows_token", op="block_rows", S=32, Hkv=8, n=131072, lo=1024, one_seq=False, Nq=1, sinks=1,
             recent=2, k=29),
        # the lists of 16 prompt tiles of 128 queries
        dict(name="block_rows_prompt", op="block_rows", S=16, Hkv=8, n=99936, lo=0, one_seq=True, Nq=128, sinks=1,
             recent=3, k=60),
        # one token of each of 32 sequences over 32 blocks for each KV head
        dict(name="heads_token_bf16", op="heads", kv="bf16", q="bf16", S=32, Nq=1, Hq=32, Hkv=8, D=128, n=8192,
             one_seq=False, blocks=32, prefill=False),
        # 16 prompt tiles of 128 queries over 64 blocks for each KV head, causal
        dict(name="heads_prompt_bf16", op="heads", kv="bf16", q="bf16", S=16, Nq=128, Hq=32, Hkv=8, D=128, n=16384,
             one_seq=True, blocks=64, prefill=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["weights", "weights", "evict", "bounds", "scores", "block_rows", "heads", "heads"])
    Hq, Hkv = rng.choice([(32, 8), (16, 2), (8, 8), (32, 4), (8, 2), (64, 8)])
    q = rng.choice(["bf16", "f16"])
    if op == "weights":
        kv = rng.choice([q, q, "i8", "i4", "f8"])
        D = rng.choice([64, 128, 128, 256])
        Nq = _log(rng, 1, 1024) if rng.random() < 0.5 else 1
        n = _log(rng, 17, 65536)
        Nq = max(1, min(Nq, n, int(2.4e11 / (2 * n * Hq * D))))
        S = min(_log(rng, 1, 32), max(1, (1 << 28) // (n * Nq * Hq)), max(1, 262144 // n))
        return dict(op=op, kv=kv, q=q, S=S, Nq=Nq, Hq=Hq, Hkv=Hkv, D=D, n=n, ragged=rng.random() < 0.5,
                    layout=rng.choice(["shuffled", "pages", "runs"]), causal=Nq > 1)
    if op == "evict":
        n = _log(rng, 100, 131072)
        S = min(_log(rng, 1, 32), max(1, 400000 // n))
        keep = rng.randint(n // 16 + 3, n)
        sinks = rng.randint(0, 2)
        recent = rng.randint(0, (keep - sinks) // 2)
        return dict(op=op, S=S, Hkv=Hkv, n=n, L=n + rng.randint(0, 40), ragged=rng.random() < 0.5, sinks=sinks,
                    recent=recent, k=keep - sinks - recent)
    if op == "bounds":
        pages = _log(rng, 1, 2000)
        kv = rng.choice([q, q, "i8", "i4", "f8"])
        return dict(op=op, kv=kv, q=q, Hkv=Hkv, D=rng.choice([64, 128, 256]), pages=pages,
                    pool_pages=pages + rng.randint(0, 200), full=rng.random() < 0.5)
    one = rng.random() < 0.4
    if op == "scores":
        Nq = rng.randint(2, 128) if one else rng.choice([1, 1, 1, 2, 4])
        n = _log(rng, max(200, 2 * Nq), 131072)
        return dict(op=op, q=q, S=_log(rng, 1, 12 if one else 32), Nq=Nq, Hq=Hq, Hkv=Hkv, D=rng.choice([64, 128, 256]),
                    n=n, lo=0 if one else max(1, n // rng.randint(1, 100)), one_seq=one)
    if op == "block_rows":
        Nq = rng.randint(2, 128) if one else 1
        n = _log(rng, max(200, 2 * Nq), 131072)
        return dict(op=op, S=_log(rng, 1, 12 if one else 32), Hkv=Hkv, n=n, lo=0 if one else max(1, n // rng.randint(1, 100)),
                    one_seq=one, Nq=Nq, sinks=rng.randint(0, 2), recent=rng.randint(1, 4), k=rng.randint(0, 100))
    prefill = rng.random() < 0.4
    blocks = rng.randint(4, 48)
    n = PAGE * (blocks + rng.randint(1, 100)) - rng.randint(0, PAGE - 1)
    if prefill:
        return dict(op=op, kv=q, q=q, S=_log(rng, 1, 12), Nq=rng.randint(9, 128), Hq=Hq, Hkv=Hkv, D=128, n=n,
                    one_seq=True, blocks=blocks, prefill=True)
    kv = rng.choice([q, q, "i8", "i4", "f8"])
    return dict(op=op, kv=kv, q=q, S=_log(rng, 1, 32), Nq=1 if Hq // Hkv > 4 else rng.choice([1, 1, 2]), Hq=Hq, Hkv=Hkv,
                D=128, n=n, one_seq=False, blocks=blocks, prefill=False)


def _lens(c):
    """Entries of each slice: fixed by the case, so that the work is too."""
    S, n = c["S"], c["n"]
    if c.get("one_seq"):   # consecutive query tiles of one sequence of n tokens
        return [n - (S - 1 - s) * c["Nq"] if n - (S - 1 - s) * c["Nq"] >= c["Nq"] else n for s in range(S)]
    lo = c["lo"] if "lo" in c else (max(1, n // 16, c.get("Nq", 1)) if c.get("ragged") else n)
    return [n - int((n - lo) * (1.0 - (lo / n) ** (s / max(1, S - 1))) / max(1e-9, 1.0 - lo / n)) if lo < n else n
            for s in range(S)]


# ---------------------------------------------------------------------------
# inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _pool(c, g, R):
    """One pool tensor and its scales (None for a 16-bit pool)."""
    Hkv, D, kv = c["Hkv"], c["D"], c["kv"]
    if kv in _TYPES:
        return _normal(g, (R, Hkv, D), _TYPES[kv]), None
    x = torch.randn((R, Hkv, D), generator=g, device="cuda")
    scale = (torch.rand((R // PAGE, Hkv, PAGE), generator=g, device="cuda") * 0.5 + 0.75)
    if kv == "i8":
        return (x * 40).round().clamp(-127, 127).to(torch.int8), (scale / 40).half()
    if kv == "f8":
        return (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn), (scale / 100).half()
    n4 = (x * 3).round().clamp(-7, 7).to(torch.int32) & 15
    return (n4[..., 0::2] | (n4[..., 1::2] << 4)).to(torch.uint8), (scale / 3).half()


def _row_lists(c, g, lens, L, R):
    """[S, L] pool rows, every one in at most one list; -1 past a slice's entries."""
    S = c["S"]
    total = sum(lens)
    if c["layout"] == "shuffled":
        flat = torch.randperm(R, generator=g, device="cuda")[:total]
    elif c["layout"] == "runs":
        flat = torch.arange(total, device="cuda")
    else:
        pages = torch.randperm(R // PAGE, generator=g, device="cuda")
        flat = (pages[:, None] * PAGE + torch.arange(PAGE, device="cuda")).reshape(-1)
    rows = torch.full((S, L), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, m in enumerate(lens):
        rows[s, :m] = flat[at:at + m].to(torch.int32)
        at += m if c["layout"] != "pages" else -(-m // PAGE) * PAGE
    return rows


def _page_tables(c, g, lens):
    """Page tables of the case's sequences, the sequence of each slice, and the pages of the pool."""
    S = c["S"]
    held = [c["n"]] if c["one_seq"] else lens
    counts = [-(-m // PAGE) for m in held]
    perm = torch.randperm(sum(counts), generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(held), max(counts)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, m in enumerate(counts):
        table[i, :m] = perm[at:at + m]
        at += m
    seq = torch.zeros(S, dtype=torch.int32, device="cuda") if c["one_seq"] else None
    return table, seq, sum(counts)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = dict(c=c)
    if c["op"] == "weights":
        lens = _lens(c)
        S, L = c["S"], max(lens)
        R = -(-sum(-(-m // PAGE) * PAGE for m in lens) // PAGE) * PAGE
        st["k"], st["k_scale"] = _pool(c, g, R)
        st["q"] = _normal(g, (S, c["Nq"], c["Hq"], c["D"]), _TYPES[c["q"]])
        st["rows"] = _row_lists(c, g, lens, L, R)
        st["lens"] = _ints(lens)
        st["scale"] = 1.0 / math.sqrt(c["D"])
        # what an attention call over these lists returned beside its output
        x = _logits(st["q"], _gather(c, st["k"], st["k_scale"], st["rows"]), st["scale"])
        x.masked_fill_(~_visible(c, st["rows"], st["lens"]), -math.inf)
        lse = torch.logsumexp(x, dim=-1)
        del x
        st["lse"] = lse.reshape(S, c["Hkv"], c["Nq"], -1).transpose(1, 2).reshape(S, c["Nq"], c["Hq"]).contiguous()
        # totals of about one earlier step
        st["acc"] = torch.rand((S, c["Hkv"], L), generator=g, device="cuda") * (c["Nq"] * c["Hq"] / c["Hkv"] / c["n"])
    elif c["op"] == "evict":
        lens = _lens(c)
        S, L = c["S"], c["L"]
        # attention weight gathers on few entries: log-normal totals
        st["acc"] = torch.exp(2.0 * torch.randn((S, c["Hkv"], L), generator=g, device="cuda"))
        st["rows"] = torch.full((S, L), -1, dtype=torch.int32, device="cuda")
        perm = torch.randperm(sum(lens), generator=g, device="cuda").to(torch.int32)
        at = 0
        for s, m in enumerate(lens):
            st["rows"][s, :m] = perm[at:at + m]
            at += m
        st["lens"] = _ints(lens)
    elif c["op"] == "bounds":
        P, T = c["pages"], _TYPES[c["q"]]
        st["k"], st["k_scale"] = _pool(c, g, c["pool_pages"] * PAGE)
        st["pages"] = torch.randperm(c["pool_pages"], generator=g, device="cuda")[:P].to(torch.int32)
        fill = torch.randint(1, PAGE + 1, (P,), generator=g, device="cuda").to(torch.int32)
        if c["full"]:
            fill[:-1] = PAGE
        st["fill"] = fill
        st["kmin"] = torch.zeros((c["pool_pages"], c["Hkv"], c["D"]), dtype=T, device="cuda")
        st["kmax"] = torch.zeros_like(st["kmin"])
    elif c["op"] == "scores":
        lens = _lens(c)
        T = _TYPES[c["q"]]
        st["table"], st["seq"], pages = _page_tables(c, g, lens)
        st["lens"] = _ints(lens)
        st["q"] = _normal(g, (c["S"], c["Nq"], c["Hq"], c["D"]), T)
        mid, half = (torch.randn((pages, c["Hkv"], c["D"]), generator=g, device="cuda") for _ in range(2))
        st["kmin"], st["kmax"] = (0.5 * mid - 2 - half.abs()).to(T), (0.5 * mid + 2 + half.abs()).to(T)
    elif c["op"] == "block_rows":
        lens = _lens(c)
        st["table"], st["seq"], _ = _page_tables(c, g, lens)
        st["lens"] = _ints(lens)
        NB = st["table"].shape[1]
        st["score"] = 30 + 4 * torch.randn((c["S"], c["Hkv"], NB), generator=g, device="cuda")
        held = (st["lens"] + PAGE - 1) // PAGE
        st["score"].masked_fill_(torch.arange(NB, device="cuda")[None, None] >= held[:, None, None], -math.inf)
    else:   # heads
        lens = _lens(c)
        S, Hkv, B = c["S"], c["Hkv"], c["blocks"]
        table, seq, pages = _page_tables(c, g, lens)
        st["k"], st["k_scale"] = _pool(c, g, pages * PAGE)
        st["v"], st["v_scale"] = _pool(c, g, pages * PAGE)
        st["q"] = _normal(g, (S, c["Nq"], c["Hq"], c["D"]), _TYPES[c["q"]])
        st["scale"] = 1.0 / math.sqrt(c["D"])
        st["rows"] = torch.full((S, Hkv, B * PAGE), -1, dtype=torch.int32, device="cuda")
        n_list = []
        for s, m in enumerate(lens):
            nb = -(-m // PAGE)
            recent = min(nb, 1 + -(-c["Nq"] // PAGE), B)
            pick = min(B, nb) - recent
            blk = torch.rand((Hkv, nb), generator=g, device="cuda")
            blk[:, nb - recent:] = 2.0
            blk = blk.topk(pick + recent, dim=1).indices.sort(dim=1).values
            page = table[0 if c["one_seq"] else s][blk]
            r = (page[:, :, None] * PAGE + torch.arange(PAGE, device="cuda", dtype=torch.int32)).reshape(Hkv, -1)
            keep = r.shape[1] - (nb * PAGE - m)
            st["rows"][s, :, :keep] = r[:, :keep]
            n_list.append(keep)
        st["n_list"] = n_list
        st["lens"] = _ints(n_list)[:, None].expand(S, Hkv).contiguous()
    return st


# ---------------------------------------------------------------------------
# the plain form


def _widen(c, x, scale, rows):
    """fp32 values of pool elements x of the given pool rows [..., Hkv, D]."""
    if c["kv"] in _TYPES:
        return x.float()
    if c["kv"] == "i4":
        x = x.to(torch.int32)
        x = torch.stack(((x & 15) ^ 8, (x >> 4) ^ 8), dim=-1).flatten(-2) - 8
    return x.float() * scale[rows // PAGE, :, rows % PAGE].float()[..., None]


def _gather(c, pool, scale, rows):
    """[S, Hkv, L, D] fp32 from lists [S, L]."""
    r = rows.clamp(min=0).long()
    x = pool.view(torch.uint8)[r].view(pool.dtype) if c["kv"] == "f8" else pool[r]
    return _widen(c, x, scale, r).transpose(1, 2)


def _gather_heads(c, pool, scale, rows):
    """[S, Hkv, L, D] fp32 from lists [S, Hkv, L]."""
    r = rows.clamp(min=0).long()
    g = torch.arange(c["Hkv"], device=rows.device)[None, :, None]
    x = pool.view(torch.uint8)[r, g].view(pool.dtype) if c["kv"] == "f8" else pool[r, g]
    if c["kv"] in _TYPES:
        return x.float()
    if c["kv"] == "i4":
        x = x.to(torch.int32)
        x = torch.stack(((x & 15) ^ 8, (x >> 4) ^ 8), dim=-1).flatten(-2) - 8
    return x.float() * scale[r // PAGE, g, r % PAGE].float()[..., None]


def _logits(q, k, scale):
    """q [S, Nq, Hq, D], k [S, Hkv, L, D] -> [S, Hkv, Nq * G, L]."""
    S, Nq, Hq, D = q.shape
    qh = q.float().reshape(S, Nq, k.shape[1], -1, D).transpose(1, 2).reshape(S, k.shape[1], -1, D)
    return torch.matmul(qh, k.transpose(-1, -2)).mul_(scale)


def _visible(c, rows, lens):
    """[S, 1, Nq * G, L] (lists [S, L]) or [S, Hkv, Nq * G, L] (lists [S, Hkv, L])."""
    if rows.dim() == 2:
        rows, lens = rows[:, None], lens[:, None]
    L = rows.shape[-1]
    j = torch.arange(L, device=rows.device)
    ok = (rows >= 0) & (j < lens[..., None])
    last = lens[..., None] - 1
    if c.get("causal", c.get("prefill")) and c["Nq"] > 1:
        last = lens[..., None] - c["Nq"] + torch.arange(c["Nq"], device=rows.device).repeat_interleave(c["Hq"] // c["Hkv"])
    return ok[:, :, None, :] & (j <= last[..., None])


def _weights(st):
    c = st["c"]
    S, Hkv = c["S"], c["Hkv"]
    x = _logits(st["q"], _gather(c, st["k"], st["k_scale"], st["rows"]), st["scale"])
    lse = st["lse"].reshape(S, c["Nq"], Hkv, -1).transpose(1, 2).reshape(S, Hkv, -1, 1)
    w = torch.exp(x.sub_(lse))
    w.masked_fill_(~_visible(c, st["rows"], st["lens"]), 0.0)
    st["acc"] += w.sum(dim=2)
    return st["acc"]


def _evict(st):
    c, acc, rows, lens = st["c"], st["acc"], st["rows"], st["lens"]
    S, Hkv, L = acc.shape
    budget = c["sinks"] + c["recent"] + c["k"]
    pos = torch.arange(L, device=acc.device)[None]
    live = (pos < lens[:, None]) & (rows >= 0)
    total = acc.double().sum(dim=1).float()
    n = lens[:, None]
    forced = live & ((pos < c["sinks"]) | (pos >= n - c["recent"]))
    order = torch.where(live & ~forced, total, torch.full_like(total, -math.inf))
    rank = torch.empty_like(rows, dtype=torch.int64)
    rank.scatter_(1, order.sort(dim=1, descending=True, stable=True).indices, pos.expand(S, L).contiguous())
    keep = forced | (live & ~forced & (rank < c["k"]))
    first = torch.sort((~keep).to(torch.uint8), dim=1, stable=True).indices[:, :budget]   # kept positions, in order
    if first.shape[1] < budget:
        first = torch.nn.functional.pad(first, (0, budget - first.shape[1]))
    count = keep.sum(dim=1)
    there = torch.arange(budget, device=acc.device)[None] < count[:, None]
    new_rows = torch.where(there, rows.gather(1, first), -1)
    new_acc = acc.gather(2, first[:, None].expand(S, Hkv, budget)) * there[:, None]
    drop = live & ~keep
    at = torch.sort((~drop).to(torch.uint8), dim=1, stable=True).indices
    freed = torch.where(pos < drop.sum(dim=1)[:, None], rows.gather(1, at), -1)
    return {"rows": new_rows, "len": count.to(torch.int32), "acc": new_acc, "kept": torch.where(there, first, -1).to(torch.int32),
            "freed": freed}


def _round_up(x, T):
    """The smallest value of the 16-bit type T that is not below x."""
    y = x.to(T)
    bits = y.view(torch.int16)
    above = torch.where(y > 0, bits + 1, torch.where(y < 0, bits - 1, torch.ones_like(bits)))
    return torch.where(y.float() < x, above, bits).view(T)


def _bounds(st):
    c = st["c"]
    P, page = c["pages"], st["pages"].long()
    rows = page[:, None] * PAGE + torch.arange(PAGE, device=page.device)
    k = st["k"].view(torch.uint8)[rows].view(st["k"].dtype) if c["kv"] == "f8" else st["k"][rows]
    x = _widen(c, k, st["k_scale"], rows)                     # [P, 64, Hkv, D]
    there = (torch.arange(PAGE, device=page.device)[None] < st["fill"][:, None])[:, :, None, None]
    lo = torch.where(there, x, math.inf).amin(dim=1)
    hi = torch.where(there, x, -math.inf).amax(dim=1)
    T = st["kmin"].dtype
    st["kmin"][page] = -_round_up(-lo, T)
    st["kmax"][page] = _round_up(hi, T)
    return st["kmin"], st["kmax"]


def _scores(st):
    c = st["c"]
    S, Nq, Hq, D = st["q"].shape
    Hkv, NB = c["Hkv"], st["table"].shape[1]
    seq = st["seq"].long() if st["seq"] is not None else torch.arange(S, device="cuda")
    page = st["table"][seq].long()                           # [S, NB]
    qh = st["q"].float().reshape(S, Nq, Hkv, -1, D).transpose(1, 2).reshape(S, Hkv, -1, D)
    at = page.clamp(min=0)
    hi = torch.matmul(qh.clamp(min=0), st["kmax"][at].float().permute(0, 2, 3, 1))
    lo = torch.matmul(qh.clamp(max=0), st["kmin"][at].float().permute(0, 2, 3, 1))
    best = (hi + lo).amax(dim=2)                             # [S, Hkv, NB]
    held = (st["lens"] + PAGE - 1) // PAGE
    there = (page >= 0) & (torch.arange(NB, device="cuda")[None] < held[:, None])
    return best.masked_fill(~there[:, None], -math.inf)


def _block_rows(st):
    c, score, lens = st["c"], st["score"], st["lens"]
    S, Hkv, NB = score.shape
    budget = c["sinks"] + c["recent"] + c["k"]
    seq = st["seq"].long() if st["seq"] is not None else torch.arange(S, device="cuda")
    table = st["table"][seq]
    held = ((lens + PAGE - 1) // PAGE)[:, None, None]
    b = torch.arange(NB, device="cuda")[None, None]
    forced = (b < held) & ((b < c["sinks"]) | (b >= held - c["recent"]))
    middle = (b < held) & ~forced
    order = torch.where(middle, score, -math.inf)
    rank = torch.empty((S, Hkv, NB), dtype=torch.int64, device="cuda")
    rank.scatter_(2, order.sort(dim=2, descending=True, stable=True).indices, b.expand(S, Hkv, NB).contiguous())
    keep = (forced | (middle & (rank < c["k"]))).expand(S, Hkv, NB)
    first = torch.sort((~keep).to(torch.uint8), dim=2, stable=True).indices[:, :, :budget]
    if first.shape[2] < budget:
        first = torch.nn.functional.pad(first, (0, budget - first.shape[2]))
    count = keep.sum(dim=2)
    there = torch.arange(budget, device="cuda")[None, None] < count[..., None]
    page = table[:, None].expand(S, Hkv, NB).gather(2, first)
    t = torch.arange(PAGE, device="cuda")
    inside = there[..., None] & (first[..., None] * PAGE + t < lens[:, None, None, None])
    rows = torch.where(inside & (page[..., None] >= 0), page[..., None] * PAGE + t, -1).to(torch.int32)
    return rows.reshape(S, Hkv, budget * PAGE), inside.sum(dim=(2, 3)).to(torch.int32)


def _heads(st):
    c = st["c"]
    S, Nq, Hq, D = st["q"].shape
    x = _logits(st["q"], _gather_heads(c, st["k"], st["k_scale"], st["rows"]), st["scale"])
    x.masked_fill_(~_visible(c, st["rows"], st["lens"]), -math.inf)
    m = x.amax(dim=-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - m)
    l = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, _gather_heads(c, st["v"], st["v_scale"], st["rows"])) / l.clamp(min=1e-30)
    lse = (m + torch.log(l)).reshape(S, c["Hkv"], Nq, -1).transpose(1, 2).reshape(S, Nq, Hq)
    out = o.reshape(S, c["Hkv"], Nq, -1, D).transpose(1, 2).reshape(S, Nq, Hq, D)
    return out.to(st["q"].dtype), lse


_PLAIN = {"weights": _weights, "evict": _evict, "bounds": _bounds, "scores": _scores, "block_rows": _block_rows,
          "heads": _heads}


# ---------------------------------------------------------------------------
# the library's calls


def _own(st):
    import row_indexed_flash_gb300 as far
    c = st["c"]
    if c["op"] == "weights":
        return far.fa_rows_weights(st["q"], st["k"], st["rows"], st["scale"], st["lse"], st["acc"], kv_len=st["lens"],
                                   causal=c["causal"], k_scale=st["k_scale"])
    if c["op"] == "evict":
        rows, length, acc, kept, freed = far.fa_kv_evict(st["acc"], st["rows"], st["lens"], c["sinks"], c["recent"], c["k"])
        return {"rows": rows, "len": length, "acc": acc, "kept": kept, "freed": freed}
    if c["op"] == "bounds":
        return far.fa_kv_block_bounds(st["k"], st["pages"], st["fill"], st["kmin"], st["kmax"], k_scale=st["k_scale"])
    if c["op"] == "scores":
        return far.fa_kv_block_scores(st["q"], st["kmin"], st["kmax"], st["table"], st["lens"], slice_seq=st["seq"])
    if c["op"] == "block_rows":
        return far.fa_kv_block_rows(st["score"], st["table"], st["lens"], c["sinks"], c["recent"], c["k"], slice_seq=st["seq"])
    attend = far.fa_rows_prefill_heads if c["prefill"] else far.fa_rows_decode_heads
    return attend(st["q"], st["k"], st["v"], st["rows"], st["scale"], kv_len=st["lens"], causal=c["prefill"],
                  k_scale=st["k_scale"], v_scale=st["v_scale"], out_dtype=st["q"].dtype, want_lse=True)


def run(state):
    if own:
        return _own(state)
    else:
        return _PLAIN[state["c"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without


def _row_bytes(c):
    """Bytes of one (pool row, KV head) of K or V."""
    return {"bf16": 2 * c["D"], "f16": 2 * c["D"], "i8": c["D"] + 2, "f8": c["D"] + 2, "i4": c["D"] // 2 + 2}[c["kv"]]


def work(case):
    c = case
    if c["op"] == "bounds":
        return {"bytes": c["pages"] * c["Hkv"] * (PAGE * _row_bytes(c) + 4 * c["D"]), "flops": 2 * c["pages"] * PAGE * c["Hkv"] * c["D"]}
    S, Hkv = c["S"], c["Hkv"]
    lens = _lens(c)
    if c["op"] == "weights":
        Nq, Hq, D = c["Nq"], c["Hq"], c["D"]
        seen = sum(m * Nq - (Nq * (Nq - 1) // 2 if c["causal"] else 0) for m in lens)   # (query, key) pairs
        return {"bytes": sum(lens) * (Hkv * (_row_bytes(c) + 8) + 4) + S * Nq * Hq * (2 * D + 4), "flops": 2 * D * Hq * seen}
    if c["op"] == "evict":
        keep = sum(min(m, c["sinks"] + c["recent"] + c["k"]) for m in lens)
        # totals and rows read, kept rows, positions and totals written, the dropped rows written
        return {"bytes": sum(lens) * (4 * Hkv + 4) + keep * (4 * Hkv + 8) + (sum(lens) - keep) * 4, "flops": sum(lens) * Hkv}
    if c["op"] == "scores":
        blocks = [-(-m // PAGE) for m in lens]
        read = max(blocks) if c["one_seq"] else sum(blocks)
        return {"bytes": read * (Hkv * 4 * c["D"] + 4) + sum(blocks) * Hkv * 4 + S * c["Nq"] * c["Hq"] * 2 * c["D"],
                "flops": 4 * c["D"] * c["Nq"] * c["Hq"] * sum(blocks)}
    if c["op"] == "block_rows":
        blocks = [-(-m // PAGE) for m in lens]
        keep = [min(b, c["sinks"] + c["recent"] + c["k"]) for b in blocks]
        return {"bytes": sum(blocks) * Hkv * 4 + sum(blocks) * 4 + sum(keep) * Hkv * PAGE * 4, "flops": sum(blocks) * Hkv}
    n = [min(-(-m // PAGE), c["blocks"]) * PAGE - (-m) % PAGE for m in lens]
    Nq = c["Nq"]
    seen = sum(m * Nq - (Nq * (Nq - 1) // 2 if c["prefill"] else 0) for m in n)
    rows = sum(n) if not c["one_seq"] else min(sum(n), c["n"])   # tiles of one sequence share rows
    return {"bytes": rows * Hkv * 2 * _row_bytes(c) + sum(n) * Hkv * 4 + S * Nq * c["Hq"] * (4 * c["D"] + 4),
            "flops": 4 * c["D"] * c["Hq"] * seen}


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def _f64(c, pool, scale, rows, g):
    """Values of head g of the listed pool rows, [n, D] in fp64."""
    if c["kv"] in _TYPES:
        return pool[rows, g].double()
    if c["kv"] == "i4":
        b = pool[rows, g].short()
        lo, hi = b % 16, b // 16
        both = torch.empty((len(rows), 2 * b.shape[1]), dtype=torch.float64, device=b.device)
        both[:, 0::2], both[:, 1::2] = torch.where(lo > 7, lo - 16, lo), torch.where(hi > 7, hi - 16, hi)
    else:
        both = pool[:, g].float().double()[rows]
    return both * scale[rows.div(PAGE, rounding_mode="floor"), g, rows.remainder(PAGE)].double()[:, None]


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "weights":
        acc = st["acc"].double()
        G = c["Hq"] // c["Hkv"]
        for s, m in enumerate(_lens(c)):
            rows = st["rows"][s, :m].long()
            hidden = torch.arange(m, device="cuda")[None] > (torch.arange(c["Nq"], device="cuda")[:, None] + m - c["Nq"])
            for g in range(c["Hkv"]):
                k = _f64(c, st["k"], st["k_scale"], rows, g)
                for h in range(g * G, (g + 1) * G):
                    x = st["q"][s, :, h].double() @ k.T * st["scale"] - st["lse"][s, :, h].double()[:, None]
                    if c["causal"]:
                        x[hidden] = -math.inf
                    acc[s, g, :m] += x.exp().sum(0)
        return acc
    if c["op"] == "evict":
        S, Hkv, L = st["acc"].shape
        budget = c["sinks"] + c["recent"] + c["k"]
        a = st["acc"].cpu().numpy().astype(np.float64)
        r = st["rows"].cpu().numpy()
        out = {"rows": np.full((S, budget), -1, np.int32), "len": np.zeros(S, np.int32), "acc": np.zeros((S, Hkv, budget)),
               "kept": np.full((S, budget), -1, np.int32), "freed": np.full((S, L), -1, np.int32)}
        for s, m in enumerate(_lens(c)):
            t = a[s, :, :m].sum(0).astype(np.float32)
            lo, hi = min(c["sinks"], m), max(min(c["sinks"], m), m - c["recent"])
            best = lo + np.lexsort((np.arange(lo, hi), -t[lo:hi]))[:c["k"]]
            keep = np.concatenate([np.arange(lo), np.sort(best), np.arange(hi, m)]).astype(np.int64)
            lost = np.setdiff1d(np.arange(m), keep)
            out["len"][s] = len(keep)
            out["rows"][s, :len(keep)], out["kept"][s, :len(keep)] = r[s, keep], keep
            out["acc"][s, :, :len(keep)] = a[s][:, keep]
            out["freed"][s, :len(lost)] = r[s, lost]
        return out
    if c["op"] == "bounds":
        lo, hi = st["kmin"].double(), st["kmax"].double()
        for page, fill in zip(st["pages"].tolist(), st["fill"].tolist()):
            rows = torch.arange(page * PAGE, page * PAGE + fill, device="cuda")
            if c["kv"] in _TYPES:
                x = st["k"][rows].double()
            else:
                x = torch.stack([_f64(c, st["k"][page * PAGE:(page + 1) * PAGE], st["k_scale"][page:page + 1],
                                      rows - page * PAGE, g) for g in range(c["Hkv"])], dim=1)
            lo[page], hi[page] = x.min(0).values, x.max(0).values
        return lo, hi
    if c["op"] == "scores":
        S, NB = c["S"], st["table"].shape[1]
        score = torch.full((S, c["Hkv"], NB), -math.inf, dtype=torch.float64, device="cuda")
        G = c["Hq"] // c["Hkv"]
        for s, m in enumerate(_lens(c)):
            page = st["table"][0 if c["one_seq"] else s, :-(-m // PAGE)].long()
            for h in range(c["Hq"]):
                q = st["q"][s, :, h].double()
                up = torch.where(q > 0, q, 0.0) @ st["kmax"][page, h // G].double().T
                down = torch.where(q < 0, q, 0.0) @ st["kmin"][page, h // G].double().T
                at = score[s, h // G, :len(page)]
                at.copy_(torch.maximum(at, (up + down).max(0).values))
        return score
    if c["op"] == "block_rows":
        S, Hkv, NB = st["score"].shape
        budget = c["sinks"] + c["recent"] + c["k"]
        sc, pt = st["score"].cpu().numpy(), st["table"].cpu().numpy()
        rows, length = np.full((S, Hkv, budget * PAGE), -1, np.int32), np.zeros((S, Hkv), np.int32)
        for s, m in enumerate(_lens(c)):
            nb = -(-m // PAGE)
            lo, hi = min(c["sinks"], nb), max(min(c["sinks"], nb), nb - c["recent"])
            for g in range(Hkv):
                best = lo + np.lexsort((np.arange(lo, hi), -sc[s, g, lo:hi]))[:c["k"]]
                keep = np.concatenate([np.arange(lo), np.sort(best), np.arange(hi, nb)]).astype(np.int64)
                pos = (keep[:, None] * PAGE + np.arange(PAGE)).reshape(-1)
                r = (pt[0 if c["one_seq"] else s][keep][:, None] * PAGE + np.arange(PAGE)).reshape(-1)[pos < m]
                rows[s, g, :len(r)], length[s, g] = r, len(r)
        return rows, length
    # heads
    S, Nq, Hq, D = st["q"].shape
    out = torch.zeros((S, Nq, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((S, Nq, Hq), -math.inf, dtype=torch.float64, device="cuda")
    G = Hq // c["Hkv"]
    for s, m in enumerate(st["n_list"]):
        for h in range(Hq):
            rows = st["rows"][s, h // G, :m].long()
            x = st["q"][s, :, h].double() @ _f64(c, st["k"], st["k_scale"], rows, h // G).T * st["scale"]
            if c["prefill"]:
                x[torch.arange(m, device="cuda")[None] > (torch.arange(Nq, device="cuda")[:, None] + m - Nq)] = -math.inf
            lse[s, :, h] = torch.logsumexp(x, dim=1)
            out[s, :, h] = torch.softmax(x, dim=1) @ _f64(c, st["v"], st["v_scale"], rows, h // G)
    return out, lse
