"""gemm_fp8 with every remainder of k and of the outputs, in rows whose padding holds NaN, on every tile; outputs in the
middle of other values."""
import pytest
import torch

import shape_driven_tile_gb300 as sdt
from _fp8 import E4M3, assert_near, fp8_values, product, scale_values

pytestmark = pytest.mark.gpu
TILES = [16, 32, 64, 128, 192, 256]


def padded(rows, k, seed):
    """[rows, k] values in rows of a multiple of 16 (at least one more), the rest NaN."""
    whole = torch.full((rows, k // 16 * 16 + 16), 0x7F, dtype=torch.uint8, device="cuda")
    whole[:, :k] = fp8_values((rows, k), seed).view(torch.uint8)
    return whole.view(E4M3)[:, :k]


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("k", [1, 7, 16, 17, 100, 127, 129, 255, 1000, 1153])
def test_any_k(cuda_device, tile, k):
    m, n = 35, 200
    a, w = padded(m, k, 1), padded(n, k, 2)
    kb = -(-k // 128)
    sa, sw = scale_values((m, kb), 3), scale_values((2, kb), 4)
    got = sdt.gemm_fp8(a, sa, w, sw, tile=tile, out_dtype=torch.float32)
    sdt.check_device_status()
    want, slack = product(a, sa, w, sw)
    assert_near(got, want, slack)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("m,n", [(1, 8), (2, 24), (31, 120), (129, 136), (257, 264), (300, 200)])
def test_any_sizes_write_nothing_else(cuda_device, tile, m, n, out):
    k = 400
    a, w = padded(m, k, 1), padded(n, k, 2)
    sa, sw = scale_values((m, 4), 3), scale_values((-(-n // 128), 4), 4)
    rows = torch.full((m + 2, n + 16), 7.0, dtype=out, device=cuda_device)
    c = rows[1:m + 1, 8:8 + n]
    sdt.gemm_fp8(a, sa, w, sw, c, tile=tile)
    sdt.check_device_status()
    want, slack = product(a, sa, w, sw)
    assert_near(c, want, slack)
    rows[1:m + 1, 8:8 + n] = 7.0
    assert (rows == 7).all()
