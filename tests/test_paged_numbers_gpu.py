"""The paged calls' own numbers: what is no integer or number, or passes its range, is refused by name."""
import numpy as np
import pytest
import torch

import shape_driven_tile_gb300 as sdt

pytestmark = pytest.mark.gpu


@pytest.fixture
def args(cuda_device):
    i32 = dict(dtype=torch.int32, device=cuda_device)
    cache = sdt.PagedCache(*(torch.ones(4, 16, 2, 64, dtype=torch.bfloat16, device=cuda_device) for _ in range(2)))
    tables = (torch.zeros(2, **i32), torch.ones(2, **i32), torch.arange(4, **i32), torch.zeros(2, 3, **i32))
    attn = (torch.ones(2, 4, 64, dtype=torch.bfloat16, device=cuda_device), cache, tables[3], torch.ones(2, **i32))
    return tables, attn, torch.empty(2, dtype=torch.int64, device=cuda_device), sdt.paged_attn_workspace(4, 2, 64)


def test_what_is_no_number(args):
    tables, attn, slots, ws = args
    for bad in (16.0, "16", None, [16], np.float32(16)):
        with pytest.raises(TypeError, match="page_size"):
            sdt.paged_tables(*tables, page_size=bad, slots=slots)
        with pytest.raises(TypeError, match="window"):
            sdt.paged_attn_m1(*attn, workspace=ws, window=bad)
    for bad in ("1", [1.0], 1j):
        with pytest.raises(TypeError, match="scale"):
            sdt.paged_attn_m1(*attn, workspace=ws, scale=bad)


def test_what_passes_its_range(args):
    tables, attn, slots, ws = args
    for bad in (2 ** 63, -2 ** 70):
        with pytest.raises(ValueError, match="page_size"):
            sdt.paged_tables(*tables, page_size=bad, slots=slots)
        with pytest.raises(ValueError, match="window"):
            sdt.paged_attn_m1(*attn, workspace=ws, window=bad)
    with pytest.raises(ValueError, match="scale"):
        sdt.paged_attn_m1(*attn, workspace=ws, scale=1e39)


def test_other_kinds_of_the_same_numbers(args):
    tables, attn, slots, ws = args
    assert sdt.paged_tables(*tables, page_size=np.int64(16), slots=slots)[2].tolist() == [0, 16]
    want = sdt.paged_attn_m1(*attn, workspace=ws, window=1, scale=1.0)
    assert torch.equal(sdt.paged_attn_m1(*attn, workspace=ws, window=np.int32(1), scale=1), want)
    assert torch.equal(sdt.paged_attn_m1(*attn, workspace=ws, window=True, scale=np.float64(1)), want)
