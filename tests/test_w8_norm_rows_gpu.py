"""rms_norm_fp8 of many rows: CTAs that take several of them, or several groups of short ones, one after another."""
import pytest
import torch

import shape_driven_tile_gb300 as sdt
from _fp8 import assert_near, assert_quantised

pytestmark = pytest.mark.gpu


def rows(t, d, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn((t, d), generator=g, device="cuda")).to(dtype)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("also", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("t,width", [(40000, 64), (20001, 392), (20000, 1000), (2003, 4096), (400, 16392), (1300, 16392), (1301, 8128)])
def test_every_row(cuda_device, t, width, dtype, residual, also, wide):
    x, w = rows(t, width, dtype, t + width), rows(1, width, torch.float32 if wide else dtype, 7)[0]
    r = rows(t, width, dtype, 8, scale=4.0) if residual else None
    v = (x.float() + r.float()).to(dtype) if residual else x
    out = torch.empty_like(x) if also else None
    q, s = sdt.rms_norm_fp8(x, w, r, eps=1e-5, out=out)
    if residual:
        assert torch.equal(r, v)
    # a sum of `width` squares in fp32, its root (rsqrt is good to 2 steps), two products
    slack = (width / 8 + 8 + 8) * 2.0 ** -24
    for lo in range(0, t, 4096):
        part = slice(lo, lo + 4096)
        y = v[part].double()
        y = y * w.double() / torch.sqrt(y.square().mean(1, keepdim=True) + 1e-5)
        assert_quantised(q[part], s[part], y, slack)
        if also:
            assert_near(out[part], y, slack * y.abs())
