"""NaN and infinities in the cache: in values, scales and keys of a request's own tokens, and in what it does not name."""
import pytest
import torch

import shape_driven_tile_gb300 as sdt

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
INF, NAN = float("inf"), float("nan")
N, PAGE, HKV, D = 600, 16, 2, 128


def make(dev, dtype, q8):
    g = torch.Generator(device=dev).manual_seed(0)
    pages = -(-N // PAGE) + 1
    if q8:
        kv = [torch.randint(-100, 101, (pages, PAGE, HKV, D), generator=g, device=dev, dtype=torch.int8) for _ in range(2)]
        kv += [(torch.rand(pages, PAGE, HKV, D // 32, generator=g, device=dev) * 0.01 + 0.01).half() for _ in range(2)]
    else:
        kv = [torch.randn(pages, PAGE, HKV, D, generator=g, device=dev).to(dtype) for _ in range(2)]
    q = torch.randn(2, 8, D, generator=g, device=dev).to(dtype)
    return kv, q


def run(kv, q):
    dev = q.device
    pages = -(-N // PAGE)
    table = torch.stack([torch.arange(pages), torch.arange(pages)]).to(torch.int32).to(dev)
    lens = torch.tensor([N, 100], dtype=torch.int32, device=dev)
    lse = torch.empty(2, 8, device=dev)
    out = sdt.paged_attn_m1(q, sdt.PagedCache(*kv), table, lens, lse=lse, workspace=sdt.paged_attn_workspace(8, HKV, D))
    sdt.check_device_status()
    return out, lse


@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("token", [0, 333, N - 1])
def test_a_value_spoils_its_column_only(cuda_device, token, q8, dtype, bad):
    """Token 333 is only in the first request; a value of key head 1 is no matter of key head 0."""
    kv, q = make(cuda_device, dtype, q8)
    want, want_lse = run(kv, q)
    kv = [t.clone() for t in kv]
    if q8:
        kv[3][token // PAGE, token % PAGE, 1, 2] = bad
        columns = torch.arange(D, device=cuda_device) // 32 == 2
    else:
        kv[1][token // PAGE, token % PAGE, 1, 70] = bad
        columns = torch.arange(D, device=cuda_device) == 70
    got, lse = run(kv, q)
    assert torch.equal(lse, want_lse)
    hit = torch.zeros_like(got, dtype=torch.bool)
    for b, n in enumerate((N, 100)):
        hit[b, 4:] = columns if token < n else False
    assert torch.equal(got[~hit], want[~hit])
    assert not got[hit].isfinite().any()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("q8", [False, True])
def test_a_key_of_nan_is_nan_for_its_head(cuda_device, q8, dtype):
    kv, q = make(cuda_device, dtype, q8)
    want, _ = run(kv, q)
    kv = [t.clone() for t in kv]
    (kv[2] if q8 else kv[0])[333 // PAGE, 333 % PAGE, 0] = NAN
    got, lse = run(kv, q)
    assert got[0, :4].isnan().all() and lse[0, :4].isnan().all()
    assert torch.equal(got[0, 4:], want[0, 4:]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("bad", [INF, NAN])
@pytest.mark.parametrize("q8", [False, True])
def test_what_no_request_names(cuda_device, q8, bad):
    kv, q = make(cuda_device, BF16, q8)
    want, _ = run(kv, q)
    kv = [t.clone() for t in kv]
    for t in kv[2:] if q8 else kv:  # behind the longest request in its last page, and the page that none has
        t[N // PAGE, N % PAGE:] = bad
        t[-1] = bad
    got, _ = run(kv, q)
    assert torch.equal(got, want)
