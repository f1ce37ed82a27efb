"""Inputs, 64-bit references and bounds shared by the paged cache's tests (CPU, double).

Bounds, derived from the arithmetic that the operators state (u: half a unit in the last
place of the output type, relative: 2^-9 bf16, 2^-12 fp16 rounded up to 2^-8 and 2^-11 to
cover the second rounding of a value near a tie):

  score   D products summed in fp32 in any order: at most D * 2^-23 * sum_d |q_d k_d| *
          scale, times log2(e) and back; scaling and the power of two add at most
          2^-21 * (1 + |score|).  q8 adds the scale's product, one more rounding a group.
          Together dS = (D + 8) * 2^-23 * max_n(sum_d |q_d k_nd|) * scale
                        + 2^-20 * (1 + max|score|).
  output  a relative error e^dS - 1 <= 2 dS (dS <= 1/2) of every weight and of their sum
          moves sum p v by at most 4 dS * sum p |v|; weights as two 16-bit parts leave
          2^-16 (bf16, and fp16 above its subnormals) of each and, in fp16, 2^-25 of the
          largest weight; the fp32 sums of N terms N * 2^-23; then the output's rounding.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def make_cache(pages, page, heads, d, dtype, layout, seed, q8=False, device="cpu"):
    """(k, v, k_scales, v_scales), logical [pages, page, heads, d], all of it NaN or, in int8, 127 with NaN scales."""
    def empty(width, dt, fill):
        if layout == "head":
            return torch.full((pages, heads, page, width), fill, dtype=dt, device=device).transpose(1, 2)
        return torch.full((pages, page, heads, width), fill, dtype=dt, device=device)

    nan = float("nan")
    if not q8:
        return empty(d, dtype, nan), empty(d, dtype, nan), None, None
    return (empty(d, torch.int8, 127), empty(d, torch.int8, 127), empty(d // 32, torch.float16, nan),
            empty(d // 32, torch.float16, nan))


def fill(cache, table, lens, seed, dtype, spread=1.0):
    """Random keys and values at the tokens that table and lens name; nothing else is touched."""
    g = torch.Generator().manual_seed(seed)
    k, v, ks, vs = cache
    page = k.shape[1]
    for b, n in enumerate(lens):
        pos = torch.arange(n)
        at, off = table[b].long()[pos // page], pos % page
        shape = (n, *k.shape[2:])
        for x, s in ((k, ks), (v, vs)):
            if s is None:
                x[at, off] = (torch.randn(shape, generator=g) * spread).to(dtype)
            else:
                x[at, off] = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)
                s[at, off] = (torch.rand((*shape[:2], shape[2] // 32), generator=g) * 0.03 * spread + 1e-3).half()


def tables(lens, page, seed, extra=3, wide=None):
    """(table int32 [B, wide] of scattered pages, unused entries -1; number of pages of the pool)."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pool = sum(need) + extra
    ids = torch.randperm(pool, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need)) if wide is None else wide), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, pool


def numbers(x, s):
    return x.double() if s is None else x.double() * s.double().repeat_interleave(32, -1)


def attention(q, cache, table, lens, window=0, scale=None):
    """(out, lse, bound of out, bound of lse), all double [B, Hq, ...], from the definition."""
    k, v, ks, vs = cache
    B, Hq, D = q.shape
    Hkv, page = k.shape[2], k.shape[1]
    G = Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.zeros(B, Hq, D, dtype=torch.float64)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    fp16 = q.dtype is torch.float16
    for b, n in enumerate(lens):
        pos = torch.arange(max(0, n - window) if window else 0, n)
        if not len(pos):
            continue
        at, off = table[b].long()[pos // page], pos % page
        kk = numbers(k[at, off], None if ks is None else ks[at, off])
        vv = numbers(v[at, off], None if vs is None else vs[at, off])
        for i in range(Hq):
            x, y, qi = kk[:, i // G], vv[:, i // G], q[b, i].double()
            s = x @ qi * scale
            m = s.max()
            w = torch.exp(s - m)
            p = w / w.sum()
            out[b, i], lse[b, i] = p @ y, m + torch.log(w.sum())
            ds = ((D + 8) * 2.0 ** -23 * (x.abs() @ qi.abs()).max() * abs(scale) + 2.0 ** -20 * (1 + s.abs().max())).item()
            assert ds <= 0.5, "the bounds hold for small score errors only"
            a = p @ y.abs()
            tol[b, i] = (U[q.dtype] * out[b, i].abs() + (4 * ds + 2.0 ** -16 + len(pos) * 2.0 ** -23) * a
                         + (2.0 ** -25 * (y.abs().sum(0) / w.sum() + 1) if fp16 else 0))
            tol_lse[b, i] = 2 * ds + len(pos) * 2.0 ** -23 + 2.0 ** -21 * (1 + lse[b, i].abs())
    return out, lse, tol, tol_lse


def assert_within(got, want, tol, what=""):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all() or not torch.isfinite(want).all(), f"{what}: non-finite output"
    bad = ~((got - want).abs() <= tol) & ~(got == want)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst error / bound "
                           f"{((got - want).abs() / tol.clamp(min=1e-300))[bad].max():.3g}")
