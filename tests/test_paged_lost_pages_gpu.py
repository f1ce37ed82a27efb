"""Page ids outside the cache: reported, and NaN for the requests that name them, never an answer that
could be taken for one; the other requests are untouched."""
import pytest
import torch

import _paged
import shape_driven_tile_gb300 as sdt

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
BAD = (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31)


def lose(dev, lens, lost, Hq, Hkv, D, page, dtype=BF16, q8=False, layout="token", window=0, seed=0, scale=None):
    """lost: (request, page of it) whose table entries are bad, all of them inside the requests' tokens."""
    table, pool = _paged.tables(lens, page, seed)
    cache = _paged.make_cache(pool, page, Hkv, D, dtype, layout, seed, q8)
    _paged.fill(cache, table, lens, seed + 1, dtype)
    q = torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(seed + 2)).to(dtype)
    bad = table.clone()
    for i, (b, j) in enumerate(lost):
        bad[b, j] = BAD[i % len(BAD)]
    on = [None if t is None else (t.transpose(1, 2).to(dev).transpose(1, 2) if not t.is_contiguous() else t.to(dev)) for t in cache]
    handle, ws = sdt.PagedCache(*on), sdt.paged_attn_workspace(Hq, Hkv, D)
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    lse = torch.empty(len(lens), Hq, device=dev)
    hit = sorted({b for b, _ in lost})
    rest = [b for b in range(len(lens)) if b not in hit]
    good = sdt.paged_attn_m1(q.to(dev), handle, table.to(dev), n, workspace=ws, window=window, scale=scale)
    sdt.check_device_status()
    for _ in range(2):
        got = sdt.paged_attn_m1(q.to(dev), handle, bad.to(dev), n, workspace=ws, lse=lse, window=window, scale=scale)
        with pytest.raises(sdt.SdtError, match="page"):
            sdt.check_device_status()
        assert got[hit].isnan().all() and lse[hit].isnan().all()
        assert torch.equal(got[rest], good[rest])
        assert not ws[: 1 << 20].any()
    again = sdt.paged_attn_m1(q.to(dev), handle, table.to(dev), n, workspace=ws, window=window, scale=scale)
    sdt.check_device_status()
    assert torch.equal(good, again) and good.isfinite().all()


LENS = [200, 64, 1, 129, 48, 0, 77]
LOST = [(0, 0), (0, 3), (0, 12), (1, 1), (1, 2), (2, 0), (3, 8)]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_lost_pages(cuda_device, D, dtype, q8):
    lose(cuda_device, LENS, [x for x in LOST if x != (1, 2)] + [(1, 3)], 4, 2, D, 16, dtype, q8, seed=D)


@pytest.mark.parametrize("lost", [(0, 0), (0, 6), (0, 12), (2, 0), (3, 8), (6, 4)])
def test_one_lost_page(cuda_device, lost):
    lose(cuda_device, LENS, [lost], 4, 2, 64, 16)


@pytest.mark.parametrize("D", [8, 40, 80, 192])
def test_lost_pages_of_odd_widths(cuda_device, D):
    lose(cuda_device, LENS, [(0, 1), (3, 0)], 4, 2, D, 16, seed=D)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("group", [9, 24, 40, 64])
@pytest.mark.parametrize("D", [64, 256])
def test_lost_pages_of_warps_that_share_keys(cuda_device, D, group, q8):
    lose(cuda_device, LENS, [(0, 2), (0, 7), (3, 8), (6, 0)], group, 1, D, 16, BF16, q8, "head", seed=group)


@pytest.mark.parametrize("page", [1, 7, 20, 64])
def test_lost_pages_of_other_sizes(cuda_device, page):
    lose(cuda_device, [150, 33, 90], [(0, 149 // page), (1, (32 // page) // 2)], 4, 2, 64, page, seed=page)


def test_lost_pages_in_and_before_a_window(cuda_device):
    lose(cuda_device, LENS, [(0, 11), (3, 8)], 4, 2, 64, 16, window=40)
    table, pool = _paged.tables([200], 16, 0)
    cache = _paged.make_cache(pool, 16, 2, 64, BF16, "token", 0)
    _paged.fill(cache, table, [200], 1, BF16)
    q = torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(2)).to(BF16)
    table[0, :10] = -1  # pages that the window has left behind may be gone
    out = sdt.paged_attn_m1(q.to(cuda_device), sdt.PagedCache(*(t.to(cuda_device) for t in cache[:2])), table.to(cuda_device),
                            torch.tensor([200], dtype=torch.int32, device=cuda_device), workspace=sdt.paged_attn_workspace(4, 2, 64), window=40)
    sdt.check_device_status()
    assert out.isfinite().all()


@pytest.mark.parametrize("group,D", [(8, 128), (64, 128), (1, 64)])
def test_lost_pages_of_a_split_request(cuda_device, group, D):
    lose(cuda_device, [9000, 20], [(0, 333)], group, 1, D, 16, F16)


def test_lost_pages_among_many_items(cuda_device):
    lens = [(i * 29) % 70 for i in range(256)]
    lose(cuda_device, lens, [(b, 0) for b in range(3, 256, 5) if lens[b]], 8, 8, 64, 16, F16, layout="head")


def test_a_scale_of_zero(cuda_device):
    lose(cuda_device, LENS, [(0, 5)], 4, 2, 64, 16, scale=0.0)
