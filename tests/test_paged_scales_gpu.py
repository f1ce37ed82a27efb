"""paged_attn_m1 on q8 caches whose value scales lie far apart: from fp16's smallest to its largest."""
import math

import pytest
import torch

import _paged_bounds as bounds
import shape_driven_tile_gb300 as sdt

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
PAGE = 16


def scales_apart(dev, dtype, width, scales, n=300, group=2, seed=0):
    """One key head of `width`, whose value scales of group i are scales[i % len] times 1 to 2."""
    g = torch.Generator().manual_seed(seed)
    pages = -(-n // PAGE)
    k = torch.randint(-127, 128, (pages, PAGE, 1, width), generator=g, dtype=torch.int8)
    v = torch.randint(-127, 128, (pages, PAGE, 1, width), generator=g, dtype=torch.int8)
    ks = torch.full((pages, PAGE, 1, width // 32), 0.01).half()
    some = torch.tensor([scales[i % len(scales)] for i in range(width // 32)])
    vs = (some * (1 + torch.rand(pages, PAGE, 1, width // 32, generator=g)) * 0.5).clamp(2.0 ** -24, 65504).half()
    q = torch.randn(1, group, width, generator=g).to(dtype)
    out = sdt.paged_attn_m1(q.to(dev), sdt.PagedCache(*(t.to(dev) for t in (k, v, ks, vs))),
                            torch.arange(pages, dtype=torch.int32, device=dev)[None], torch.tensor([n], dtype=torch.int32, device=dev),
                            workspace=sdt.paged_attn_workspace(group, 1, width))
    sdt.check_device_status()
    rows = lambda t: t.reshape(pages * PAGE, -1)[:n].double()
    kk, sc = rows(k) * rows(ks).repeat_interleave(32, 1), rows(vs)
    vv = rows(v) * sc.repeat_interleave(32, 1)
    for i in range(group):
        qi = q[0, i].double()
        s = kk @ qi / math.sqrt(width)
        p = torch.softmax(s, 0)
        want = p @ vv
        ds = ((width + 8) * 2.0 ** -23 * (kk.abs() @ qi.abs()).max() / math.sqrt(width) + 2.0 ** -20 * (1 + s.abs().max())
              + 2.0 ** -25 * qi.abs().max() * kk.abs().sum(1).max() / math.sqrt(width)).item()  # (bf16 queries as fp16)
        tol = bounds.tolerance(want, p, vv, dtype, ds, n, sc)
        got = out[0, i].cpu().double()
        over = want.abs() > 65504 if dtype is F16 else torch.zeros(width, dtype=torch.bool)
        bad = ~over & ~((got - want).abs() <= tol)
        assert not bad.any(), f"{int(bad.sum())} columns outside, of groups {sorted(set((bad.nonzero().flatten() // 32).tolist()))}"


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("width", [64, 128, 192, 256])
@pytest.mark.parametrize("scales", [(2.0 ** -24,), (2.0 ** -15, 2.0 ** -14), (100.0,), (60000.0,)])
def test_value_scales_of_every_size(cuda_device, dtype, width, scales):
    scales_apart(cuda_device, dtype, width, scales)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("width", [64, 128, 192, 256])
@pytest.mark.parametrize("scales", [(1.0, 2.0 ** -12), (2.0 ** -20, 1.0), (100.0, 2.0 ** -22), (30000.0, 2.0 ** -22)])
def test_groups_of_a_head_far_apart(cuda_device, dtype, width, scales):
    """A group's outputs depend on its own scales alone, however large its neighbours' are."""
    scales_apart(cuda_device, dtype, width, scales)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_scales_that_grow_along_the_context(cuda_device, dtype):
    """The exponent kept outside moves in every block; early tokens' sums move with it."""
    for step in (1.02, 1.05):
        g = torch.Generator().manual_seed(3)
        n, width = 1000, 128
        pages = -(-n // PAGE)
        k = torch.zeros(pages, PAGE, 1, width, dtype=torch.int8)
        v = torch.randint(-127, 128, k.shape, generator=g, dtype=torch.int8)
        ks = torch.ones(pages, PAGE, 1, width // 32).half()
        vs = (2.0 ** -24 * step ** torch.arange(pages * PAGE).double()).clamp(max=100.0).half().view(pages, PAGE, 1, 1).repeat(1, 1, 1, width // 32)
        q = torch.ones(1, 1, width, dtype=dtype)
        out = sdt.paged_attn_m1(q.to(cuda_device), sdt.PagedCache(*(t.to(cuda_device) for t in (k, v, ks, vs))),
                                torch.arange(pages, dtype=torch.int32, device=cuda_device)[None],
                                torch.tensor([n], dtype=torch.int32, device=cuda_device), workspace=sdt.paged_attn_workspace(1, 1, width))
        sc = vs.reshape(-1, width // 32)[:n].double()
        vv = v.reshape(-1, width)[:n].double() * sc.repeat_interleave(32, 1)
        p = torch.full((n,), 1 / n, dtype=torch.float64)
        want = p @ vv
        tol = bounds.tolerance(want, p, vv, dtype, 2.0 ** -20, n, sc)
        assert ((out[0, 0].cpu().double() - want).abs() <= tol).all()
