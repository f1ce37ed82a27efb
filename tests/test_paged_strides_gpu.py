"""paged_append of one token or one head: the stride of a dimension that never steps may be anything."""
import pytest
import torch

import shape_driven_tile_gb300 as sdt

pytestmark = pytest.mark.gpu
D, PAGE = 64, 16


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("tokens,heads,strides", [(1, 1, (67, 3, 1)), (1, 1, (0, 0, 1)), (1, 3, (1, 72, 1)), (1, 2, (199, 64, 1)),
                                                  (5, 1, (80, 5, 1)), (5, 1, (64, 1, 1))])
def test_strides_that_never_step(cuda_device, tokens, heads, strides, q8):
    g = torch.Generator(device=cuda_device).manual_seed(3)
    rows = torch.randn(4096, generator=g, device=cuda_device).to(torch.bfloat16)
    k, v = (torch.as_strided(rows, (tokens, heads, D), strides, at) for at in (0, 2048))
    kv = [torch.zeros(2, PAGE, heads, D, dtype=torch.int8 if q8 else torch.bfloat16, device=cuda_device) for _ in range(2)]
    kv += [torch.zeros(2, PAGE, heads, D // 32, dtype=torch.float16, device=cuda_device) for _ in range(2 if q8 else 0)]
    same = [torch.zeros_like(t) for t in kv]
    slots = torch.arange(tokens, device=cuda_device) * 3 + 7
    sdt.paged_append(k, v, slots, sdt.PagedCache(*kv))
    sdt.paged_append(k.contiguous().clone(), v.contiguous().clone(), slots, sdt.PagedCache(*same))
    sdt.check_device_status()
    for a, b in zip(kv, same):
        assert torch.equal(a, b) and a.any()
    if not q8:
        assert torch.equal(kv[0].flatten(0, 1)[slots], k) and torch.equal(kv[1].flatten(0, 1)[slots], v)


@pytest.mark.parametrize("tokens,heads,strides", [(2, 1, (67, 64, 1)), (1, 2, (128, 65, 1)), (2, 2, (129, 64, 1))])
def test_strides_that_step_are_still_checked(cuda_device, tokens, heads, strides):
    rows = torch.zeros(4096, dtype=torch.bfloat16, device=cuda_device)
    k = torch.as_strided(rows, (tokens, heads, D), strides)
    cache = sdt.PagedCache(*(torch.zeros(2, PAGE, heads, D, dtype=torch.bfloat16, device=cuda_device) for _ in range(2)))
    with pytest.raises(sdt.SdtError, match="strides"):
        sdt.paged_append(k, k, torch.arange(tokens, device=cuda_device), cache)
