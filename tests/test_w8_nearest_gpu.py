"""The fp8 values of quant_fp8 next to the borders of the grid: exact ties go to even."""
import pytest
import torch

import shape_driven_tile_gb300 as sdt
from _fp8 import e4m3_grid

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


def every_ratio(dtype, device="cuda"):
    """Blocks whose largest value has each of 64 leading mantissas and whose others have each mantissa of the type, some
    binary places below."""
    bits = 7 if dtype is torch.bfloat16 else 10
    mantissas = 1.0 + torch.arange(2 ** bits, device=device, dtype=torch.float64) / 2 ** bits
    tops = mantissas[:: 2 ** bits // 64]
    rest = torch.cat([mantissas * 2.0 ** -e for e in (1, 2, 5, 8)])
    pad = -rest.numel() % 127
    rest = torch.cat([rest, rest[:pad]]).view(1, -1, 127).expand(64, -1, -1)
    sign = 1.0 - 2.0 * (torch.arange(127, device=device) % 2)
    rows = torch.cat([(4 * tops)[:, None, None].expand(64, rest.shape[1], 1), 4 * rest * sign], 2)
    return rows.flatten(1).to(dtype)


def assert_nearest(q, y):
    """q are the e4m3 numbers next to 448 * y / max|y| of each block; y is exact in 64 bits, and so is whether that is a tie.
    A quotient that is no tie but within 2^-24 of one may fall on either side (it is rounded to fp32 first)."""
    blocks = torch.nn.functional.pad(y, (0, -y.shape[1] % 128)).unflatten(1, (-1, 128))
    ratio = (448 * blocks / blocks.abs().amax(2, keepdim=True)).flatten(1)[:, : y.shape[1]]
    step = torch.exp2(torch.frexp(ratio)[1].double().sub(1).clamp(min=-6) - 3)
    tie = (ratio / step).frac().abs() == 0.5
    assert tie.any()
    got, want = q.double(), e4m3_grid(ratio)
    lo, hi = (e4m3_grid((ratio + s * ratio.abs() * 2.0 ** -24).clamp(-448, 448)) for s in (-1, 1))
    wrong = tie & (got != want)
    assert not wrong.any(), f"{int(wrong.sum())} of {int(tie.sum())} ties are not at their even neighbour"
    assert ((got >= lo) & (got <= hi) | tie).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_ties_of_quant(cuda_device, dtype):
    x = every_ratio(dtype)
    q, _ = sdt.quant_fp8(x)
    assert_nearest(q, x.double())
    g = torch.Generator(device=cuda_device).manual_seed(3)
    x = torch.randn((512, 4096), generator=g, device=cuda_device).to(dtype)
    assert_nearest(sdt.quant_fp8(x)[0], x.double())


@pytest.mark.parametrize("far", [-90, 100])
def test_ties_of_quant_at_the_ends_of_the_range(cuda_device, far):
    """Blocks whose largest values are near 2^-90 and near the largest of bf16."""
    x = (every_ratio(torch.bfloat16).double() * 2.0 ** far).to(torch.bfloat16)
    if far > 0:
        x = (x.double() * 2.0 ** 24).to(torch.bfloat16)
    assert x.isfinite().all() and torch.frexp(x.abs().max().float())[1] in (127, -87)
    assert_nearest(sdt.quant_fp8(x)[0], x.double())
