"""paged_attn_m1 where weights lie far apart: one token that outweighs a long context."""
import pytest
import torch

import _paged_bounds as bounds
import shape_driven_tile_gb300 as sdt

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
D, PAGE, HEADS = 64, 16, 8


def heavy(dev, dtype, q8, n, gap, spread, group, place, batch):
    """`batch` requests over the same n cached tokens, of which the one at `place` scores `gap` above the
    others (these: normal with `spread`) and has values of zero; the others' values lie around 1.

    One product of a score is not zero, so its error is a rounding or two of the score (2^-23 each),
    its conversion to base 2 and the power's 2^-22.
    """
    g = torch.Generator(device=dev).manual_seed(n + group)
    score = torch.randn(n, HEADS, generator=g, device=dev) * spread
    score[place] = gap
    pages = -(-n // PAGE)
    k = torch.zeros(pages * PAGE, HEADS, D, dtype=torch.int8 if q8 else dtype, device=dev)
    v = torch.zeros_like(k)
    ks = vs = None
    if q8:
        ks, vs = (torch.zeros(pages * PAGE, HEADS, D // 32, dtype=F16, device=dev) for _ in range(2))
        k[:n, :, 0] = (score * 6).round().clamp(-127, 127).to(torch.int8)
        ks[:n] = 1 / 48
        v[:n] = torch.randint(40, 80, (n, HEADS, D), generator=g, device=dev).to(torch.int8)
        vs[:n] = (torch.rand(n, HEADS, D // 32, generator=g, device=dev) * 0.01 + 0.01).half()
        v[place] = 0
    else:
        k[:n, :, 0] = (score / 8).to(dtype)
        v[:n] = (1 + 0.3 * torch.randn(n, HEADS, D, generator=g, device=dev)).to(dtype)
        v[place] = 0
    q = torch.zeros(batch, HEADS * group, D, dtype=dtype, device=dev)
    q[:, :, 0] = 8
    shape = (pages, PAGE, HEADS, -1)
    cache = sdt.PagedCache(*(None if t is None else t.view(shape) for t in (k, v, ks, vs)))
    table = torch.randperm(pages, generator=g, device=dev).to(torch.int32)  # the same rows in every order
    at = (table.long()[:, None] * PAGE + torch.arange(PAGE, device=dev)).flatten()  # where token i lies, as the table names it
    for t in (k, v, ks, vs):
        if t is not None:
            t[at] = t.clone()
    lse = torch.empty(batch, HEADS * group, device=dev)
    out = sdt.paged_attn_m1(q, cache, table.repeat(batch, 1), torch.full((batch,), n, dtype=torch.int32, device=dev),
                            scale=1.0, lse=lse, workspace=sdt.paged_attn_workspace(HEADS * group, HEADS, D))
    sdt.check_device_status()
    at = at[:n]
    for h in range(HEADS):
        kk = k[at, h, 0].double() * (1 if ks is None else ks[at, h, 0].double())
        vv = v[at, h].double() * (1 if vs is None else vs[at, h].double().repeat_interleave(32, 1))
        s = kk * 8
        want_lse = torch.logsumexp(s, 0)
        p = torch.exp(s - want_lse)
        want = p @ vv
        ds = (2.0 ** -22 * (1 + s.abs().max())).item()
        # all n keys may fall to one warp
        tol = bounds.tolerance(want, p, vv, dtype, ds, n, None if vs is None else vs[at, h].double())
        got = out[:, h * group:(h + 1) * group].double()
        worst = ((got - want).abs() / tol).max().item()
        rel = ((got - want).abs() / want.abs()).max().item()
        assert worst <= 1, f"head {h}: error / bound {worst:.3g}, relative error {rel:.3g}"
        off = (lse[:, h * group:(h + 1) * group].double() - want_lse).abs().max().item()
        assert off <= 2 * ds + n * 2.0 ** -23 + 2.0 ** -22 * (1 + abs(want_lse.item()))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n,gap,spread", [(32768, 14.0, 0.0), (32768, 15.5, 0.3), (131071, 16.3, 0.0), (131071, 16.3, 0.3), (131071, 17.0, 0.3)])
def test_one_token_outweighs_a_long_context(cuda_device, dtype, q8, n, gap, spread):
    """More items than CTAs, so that whole contexts fall to one warp; the heavy token comes first."""
    heavy(cuda_device, dtype, q8, n, gap, spread, 1, 0, 64)


@pytest.mark.parametrize("place", [0, 5000, 32767])
@pytest.mark.parametrize("group", [8, 16, 40])
def test_a_heavy_token_anywhere(cuda_device, group, place):
    heavy(cuda_device, F16, False, 32768, 16.0, 0.2, group, place, 40)


@pytest.mark.parametrize("batch", [1, 3])
def test_a_heavy_token_in_a_split_request(cuda_device, batch):
    heavy(cuda_device, F16, False, 131071, 16.3, 0.1, 2, 77777, batch)
