"""Cases of the paged key-value cache operators: what is measured, over which sizes.

One decode step of a serving program calls, in this order,

  paged_tables    block tables and slot maps of the step, from the request lengths;
  paged_append    the new tokens' keys and values into the cache, at those slots;
  paged_attn_m1   attention of one new token per request over its cached keys.

``run`` computes each in plain torch operations in 32 bits (``own`` false) or with the
library's operators (``own`` true).  Sizes are generic serving shapes, and those of this
repository's decode benchmark (K = 4096, N = 12288: the fused q, k and v projection of 32
heads of 128).
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GROUP = 32  # values per scale of the q8 cache
LARGEST_ATTN = 3.0e9  # bytes of keys and values that a drawn attention case may read
LARGEST_PLAIN = 2_200_000 * 8 * 128  # padded key elements of the plain form in a drawn case


def _attn(name, **kw):
    case = dict(name=name, op="attn", batch=1, q_heads=32, kv_heads=8, head_dim=128, page=16, min_len=1, max_len=1,
                window=0, dtype="bf16", cache="same", layout="token")
    case.update(kw)
    return case


def _append(name, **kw):
    case = dict(name=name, op="append", tokens=1, kv_heads=8, head_dim=128, page=16, run=1, dtype="bf16", cache="same",
                layout="token")
    case.update(kw)
    return case


def _tables(name, **kw):
    case = dict(name=name, op="tables", batch=1, page=16, max_len=8192, chunk=1)
    case.update(kw)
    return case


def listed():
    return [
        # the first tokens of one reply: nothing to stream, the call's latency is the step's
        _attn("attn-first-token", max_len=17, min_len=17),
        # one request in the middle of its reply, all 32 heads with keys of their own (the
        # 4096 x 12288 projection's heads)
        _attn("attn-one-mha-4k", q_heads=32, kv_heads=32, min_len=4097, max_len=4097),
        # a small serving batch of ragged requests
        _attn("attn-16-ragged", batch=16, min_len=200, max_len=2500),
        # many short chats at once, 64-wide heads with keys of their own
        _attn("attn-256-short-mha", batch=256, q_heads=16, kv_heads=16, head_dim=64, min_len=1, max_len=500, dtype="fp16"),
        # one very long context: the split over the cache's length carries it
        _attn("attn-one-128k", q_heads=64, kv_heads=8, min_len=131071, max_len=131071, page=64, layout="head"),
        # full batch with contexts from short to 32k: the largest
        _attn("attn-64-to-32k", batch=64, min_len=1000, max_len=32768, page=32, dtype="fp16"),
        # the same kind of batch with the cache in 8 bits (int8 and one fp16 scale per 32)
        _attn("attn-q8-48-to-16k", batch=48, min_len=500, max_len=16000, cache="q8"),
        # 10 query heads a key head, 80-wide heads, odd page size, sliding window
        _attn("attn-window-odd", batch=33, q_heads=20, kv_heads=2, head_dim=80, page=20, min_len=100, max_len=9001,
              window=4095),
        # a decode step's new tokens, one a request
        _append("append-decode", tokens=64, kv_heads=32),
        # a chunk of prompts: long runs of tokens, cache laid out head by head, q8
        _append("append-prompts-q8", tokens=8191, page=64, run=1000, cache="q8", layout="head"),
        # a decode step of a full batch
        _tables("tables-decode", batch=256),
        # prompt chunks and decode tokens in one step
        _tables("tables-mixed", batch=1021, page=20, max_len=30000, chunk=700),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "tables"])
    if op == "tables":
        return dict(op="tables", batch=_logint(rng, 1, 1500), page=rng.choice([1, 8, 16, 20, 32, 64, 128]),
                    max_len=_logint(rng, 64, 32768), chunk=rng.choice([1, 1, _logint(rng, 2, 1000)]))
    dtype = rng.choice(["bf16", "fp16"])
    cache = rng.choice(["same", "same", "q8"])
    layout = rng.choice(["token", "head"])
    page = rng.choice([1, 8, 16, 16, 20, 32, 64, 128])
    head_dim = rng.choice([64, 128, 128, 256] if cache == "q8" else [40, 64, 72, 80, 112, 128, 128, 224, 256])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 8, 16, 32])
    if op == "append":
        return dict(op="append", tokens=min(_logint(rng, 1, 16384), 16_777_216 // (kv_heads * head_dim)),
                    kv_heads=kv_heads, head_dim=head_dim, page=page, run=_logint(rng, 1, 2000), dtype=dtype,
                    cache=cache, layout=layout)
    batch = _logint(rng, 1, 256)
    per_token = kv_heads * head_dim * (4 if cache == "same" else 2.125)
    most = min(131072, LARGEST_ATTN / (batch * per_token), LARGEST_PLAIN / (batch * kv_heads * head_dim))
    max_len = _logint(rng, 1, max(16, int(most)))
    min_len = _logint(rng, 1, max_len)
    q_heads = kv_heads * rng.choice([g for g in (1, 1, 2, 4, 5, 7, 8, 8, 10, 16, 20, 32, 64) if kv_heads * g <= 128])
    window = _logint(rng, 1, max_len) if rng.random() < 0.2 else 0
    return dict(op="attn", batch=batch, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page=page,
                min_len=min_len, max_len=max_len, window=window, dtype=dtype, cache=cache, layout=layout)


# ---- sizes that follow from a case alone --------------------------------------------------


def _spread(lo, hi, n):
    """n lengths from hi down to lo, evenly spread over their logarithm."""
    if n == 1:
        return [hi]
    return [max(lo, min(hi, int(round(math.exp(math.log(hi) + (math.log(lo) - math.log(hi)) * i / (n - 1))))))
            for i in range(n)]


def _attn_lens(case):
    return _spread(case["min_len"], case["max_len"], case["batch"])


def _tables_lens(case):
    """(cached tokens, new tokens) of each request: every eighth has a prompt chunk, every 50th idles."""
    lens = _spread(1, case["max_len"], case["batch"])
    new = [case["chunk"] - (i // 8) % max(1, case["chunk"] // 2) if i % 8 == 0 else 0 if i % 50 == 49 else 1
           for i in range(case["batch"])]
    return [0 if i % 16 == 0 and case["chunk"] > 1 else n for i, n in enumerate(lens)], new


def work(case):
    if case["op"] == "tables":
        lens, new = _tables_lens(case)
        pages = sum(-(-(a + b) // case["page"]) - -(-a // case["page"]) for a, b in zip(lens, new))
        # lengths in, lengths and starts out, a slot per new token, new pages read and written
        return {"bytes": 4 * (4 * len(lens) + 1) + 8 * sum(new) + 8 * pages, "flops": 0}
    row = case["kv_heads"] * case["head_dim"]
    cached = row * (2.0 if case["cache"] == "same" else 1.0 + 2.0 / GROUP)  # bytes of a token's keys
    if case["op"] == "append":
        return {"bytes": case["tokens"] * (2 * row * 2 + 2 * cached + 8),
                "flops": 0 if case["cache"] == "same" else 6 * case["tokens"] * row}
    seen = [min(n, case["window"]) if case["window"] else n for n in _attn_lens(case)]
    q = case["batch"] * case["q_heads"] * case["head_dim"]
    return {"bytes": 2 * cached * sum(seen) + 2 * 2 * q + 4 * sum(-(-n // case["page"]) for n in seen) + 4 * case["batch"],
            "flops": 4.0 * case["q_heads"] * case["head_dim"] * sum(seen)}


# ---- inputs -------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _empty_cache(case, pages, dtype, width):
    """[pages, page, heads, width] of either order in memory: tokens outside heads or heads outside tokens."""
    if case["layout"] == "head":
        return torch.empty((pages, case["kv_heads"], case["page"], width), dtype=dtype, device="cuda").transpose(1, 2)
    return torch.empty((pages, case["page"], case["kv_heads"], width), dtype=dtype, device="cuda")


def _fill(t, g, dtype):
    """Normal values in any order of the cache, drawn in its memory order a gigabyte at most at a time."""
    flat = torch.as_strided(t, (t.numel(),), (1,))
    for part in flat.split(1 << 28):
        part.copy_(torch.randn(part.numel(), generator=g, dtype=dtype, device="cuda"))


def _cache(case, pages, g):
    """Keys and values of `pages` pages: normal values, or in 8 bits what such values leave."""
    dtype, d = DTYPES[case["dtype"]], case["head_dim"]
    if case["cache"] == "same":
        k, v = (_empty_cache(case, pages, dtype, d) for _ in range(2))
        _fill(k, g, dtype)
        _fill(v, g, dtype)
        return dict(k=k, v=v)
    out = {}
    for n in ("k", "v"):
        q = _empty_cache(case, pages, torch.int8, d)
        flat = torch.as_strided(q, (q.numel(),), (1,))
        for part in flat.split(1 << 28):
            part.copy_((torch.randn(part.numel(), generator=g, device="cuda") * 45).round_().clamp_(-127, 127))
        s = _empty_cache(case, pages, torch.float16, d // GROUP)
        torch.as_strided(s, (s.numel(),), (1,)).copy_(
            torch.empty(s.numel(), device="cuda").uniform_(0.012, 0.035, generator=g))
        out[n], out[n + "s"] = q, s
    return out


def _order(n, g):
    return torch.randperm(n, generator=g, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case, op=case["op"], page=case["page"])
    if case["op"] == "tables":
        lens, new = _tables_lens(case)
        order = _order(len(lens), g)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")[order]
        s["new"] = torch.tensor(new, dtype=torch.int32, device="cuda")[order]
        wide = -(-(case["max_len"] + max(new)) // case["page"])
        need = sum(-(-(a + b) // case["page"]) for a, b in zip(lens, new))
        ids = _order(need + need // 10 + 8, g).to(torch.int32)
        held = (s["lens"] + case["page"] - 1) // case["page"]
        have = torch.arange(wide, device="cuda")[None] < held[:, None]
        s["table"] = torch.full((len(lens), wide), -1, dtype=torch.int32, device="cuda")
        s["table"][have] = ids[: int(held.sum())]
        s["free"] = ids[int(held.sum()):].contiguous()
        # captured steps have room for a rounded number of tokens; what is left over is -1
        s["slots"] = torch.empty(-(-sum(new) // 64) * 64, dtype=torch.int64, device="cuda")
        return s
    dtype, heads, d = DTYPES[case["dtype"]], case["kv_heads"], case["head_dim"]
    if case["op"] == "append":
        tokens, run_len = case["tokens"], case["run"]
        per = -(-run_len // case["page"])  # pages of one run of consecutive tokens
        runs = -(-tokens // run_len)
        pages = runs * per + 3
        s.update(_cache(case, pages, g))
        t = torch.arange(tokens, device="cuda")
        at = _order(pages, g)[t // run_len * per + t % run_len // case["page"]]
        s["slots"] = at * case["page"] + t % run_len % case["page"]
        # keys and values as they leave the fused projection: slices of its rows
        q = (1 if heads == 32 else 5) * heads * d
        rows = torch.randn((tokens, q + 2 * heads * d), generator=g, device="cuda").to(dtype)
        s["new_k"] = rows[:, q:q + heads * d].unflatten(1, (heads, d))
        s["new_v"] = rows[:, q + heads * d:].unflatten(1, (heads, d))
        if own:  # the cache's handle, which a program keeps as long as the cache
            import shape_driven_tile_gb300 as sdt

            s["handle"] = sdt.PagedCache(s["k"], s["v"], s.get("ks"), s.get("vs"))
        return s
    lens = _attn_lens(case)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")[_order(len(lens), g)]
    held = (s["lens"] + case["page"] - 1) // case["page"]
    total, wide = sum(-(-n // case["page"]) for n in lens), -(-max(lens) // case["page"])
    ids = _order(total + 5, g).to(torch.int32)  # requests' pages lie scattered over the pool
    s["table"] = torch.full((len(lens), wide), -1, dtype=torch.int32, device="cuda")
    s["table"][torch.arange(wide, device="cuda")[None] < held[:, None]] = ids[:total]
    s.update(_cache(case, total + 5, g))
    s["q"] = torch.randn((case["batch"], case["q_heads"], d), generator=g, device="cuda").to(dtype)
    if own:  # the cache's handle and the workspace that a program keeps for all its steps
        import shape_driven_tile_gb300 as sdt

        s["handle"] = sdt.PagedCache(s["k"], s["v"], s.get("ks"), s.get("vs"))
        s["workspace"] = sdt.paged_attn_workspace(case["q_heads"], heads, d)
    return s


# ---- the operators ------------------------------------------------------------------------


def _run_own(s):
    import shape_driven_tile_gb300 as sdt

    if s["op"] == "tables":
        kv_lens, starts, slots, used = sdt.paged_tables(s["lens"], s["new"], s["free"], s["table"], page_size=s["page"],
                                                        slots=s["slots"])
        return dict(table=s["table"], kv_lens=kv_lens, starts=starts, slots=slots, used=used)
    if s["op"] == "append":
        sdt.paged_append(s["new_k"], s["new_v"], s["slots"], s["handle"])
        return _held(s)
    return sdt.paged_attn_m1(s["q"], s["handle"], s["table"], s["lens"], window=s["case"]["window"],
                             workspace=s["workspace"])


def _held(s):
    """The cache after an append, 8-bit keys and values as the values they stand for."""
    if "ks" not in s:
        return dict(k=s["k"], v=s["v"])
    return {n: (s[n].unflatten(3, (-1, GROUP)) * s[n + "s"].float().unsqueeze(4)).flatten(3) for n in ("k", "v")}


def _plain_tables(s):
    lens, new, page, table = s["lens"], s["new"], s["page"], s["table"]
    kv_lens = lens + new
    held = (lens + page - 1) // page
    fresh = (kv_lens + page - 1) // page - held
    first = torch.cumsum(fresh, 0) - fresh
    starts = torch.zeros(lens.numel() + 1, dtype=torch.int32, device=lens.device)
    starts[1:] = torch.cumsum(new, 0)
    j = torch.arange(table.shape[1], device=lens.device)[None] - held[:, None]
    take = (first[:, None] + j).clamp(0, s["free"].numel() - 1)
    table = torch.where((j >= 0) & (j < fresh[:, None]), s["free"][take], table)
    t = torch.arange(s["slots"].numel(), device=lens.device)
    request = torch.searchsorted(starts[1:], t, right=True, out_int32=True).clamp(max=lens.numel() - 1)
    pos = (lens[request] + t - starts[request]).clamp(max=table.shape[1] * page - 1)
    slots = table[request, pos // page].long() * page + pos % page
    return dict(table=table, kv_lens=kv_lens, starts=starts, slots=torch.where(t < starts[-1], slots, -1),
                used=fresh.sum(0, keepdim=True, dtype=torch.int32))


def _plain_append(s):
    at, off = s["slots"] // s["page"], s["slots"] % s["page"]
    for n in ("k", "v"):
        x = s["new_" + n]
        if "ks" in s:
            x = x.float().unflatten(2, (-1, GROUP))
            scale = (x.abs().amax(3) * (1.0 / 127.0)).clamp(max=65504.0).half()
            s[n + "s"][at, off] = scale
            scale = scale.float().unsqueeze(3)
            x = torch.where(scale > 0, x / scale, 0.0).round().clamp(-127, 127).to(torch.int8).flatten(2)
        s[n][at, off] = x
    return _held(s)


def _plain_attn(s):
    case, lens, q = s["case"], s["lens"], s["q"]
    pages = s["table"].clamp(min=0)
    batch, heads = q.shape[0], case["kv_heads"]

    def tokens(n):  # the requests' cached rows, [batch, tokens, heads, head_dim] in 32 bits
        x = s[n][pages].float()
        if n + "s" in s:
            x = (x.unflatten(4, (-1, GROUP)) * s[n + "s"][pages].float().unsqueeze(5)).flatten(4)
        return x.flatten(1, 2)

    at = torch.arange(pages.shape[1] * s["page"], device=q.device)[None]
    seen = at < lens[:, None]
    if case["window"]:
        seen = seen & (at >= lens[:, None] - case["window"])
    grouped = q.float().unflatten(1, (heads, -1))
    score = torch.einsum("bhgd,bnhd->bhgn", grouped, tokens("k")) * (1.0 / math.sqrt(case["head_dim"]))
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(3, keepdim=True))
    out = torch.einsum("bhgn,bnhd->bhgd", p, tokens("v")) / p.sum(3, keepdim=True)
    return out.flatten(1, 2).to(q.dtype)


def run(state):
    if own:
        return _run_own(state)
    return {"tables": _plain_tables, "append": _plain_append, "attn": _plain_attn}[state["op"]](state)


# ---- the definition in 64 bits ------------------------------------------------------------


def _numbers(q, scales, group=GROUP):
    return q.double() * scales.double().repeat_interleave(group, dim=-1)


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        out = {}
        for n in ("k", "v"):
            held = s[n].double() if case["cache"] == "same" else _numbers(s[n], s[n + "s"])
            for at, x in zip(np.array_split(s["slots"].cpu().numpy(), 8), np.array_split(np.arange(case["tokens"]), 8)):
                rows = s["new_" + n][torch.from_numpy(x).cuda()].double()
                if case["cache"] == "q8":
                    parts = rows.reshape(*rows.shape[:2], -1, GROUP)
                    scale = (parts.abs().max(-1, keepdim=True).values / 127).to(torch.float16).double()
                    rows = (torch.round(parts / scale).clamp(-127, 127) * scale).reshape(rows.shape)
                where = torch.from_numpy(at).cuda()
                held[where // case["page"], where % case["page"]] = rows
            out[n] = held
        return out
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["q_heads"] // case["kv_heads"]
    for b, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - case["window"]) if case["window"] else 0
        pos = torch.arange(lo, n, device="cuda")
        page = s["table"][b].long()[pos // case["page"]]
        off = pos % case["page"]
        for h in range(case["kv_heads"]):
            if case["cache"] == "same":
                k, v = s["k"][page, off, h].double(), s["v"][page, off, h].double()
            else:
                k, v = (_numbers(s[x][page, off, h], s[x + "s"][page, off, h]) for x in ("k", "v"))
            for i in range(h * group, (h + 1) * group):
                w = torch.softmax(k @ s["q"][b, i].double() / math.sqrt(case["head_dim"]), 0)
                out[b, i] = w @ v
    return out
