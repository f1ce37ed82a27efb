"""A dimension of one never steps: its stride may be any number, the largest too (no GPU needed)."""
import pytest
import torch

import shape_driven_tile_gb300 as sdt
from shape_driven_tile_gb300 import fp8

FAR = [2 ** 63 - 1, -(2 ** 63), 2 ** 62]


def at(i):
    return 0x100000 * (i + 1)


@pytest.mark.parametrize("far", FAR)
def test_strides_of_single_rows(far):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    quant = fp8._QUANT.pack(at(0), at(1), at(2), at(3), 1, 128, far, far, far, far, far, 1, 1)
    norm = fp8._NORM.pack(at(0), at(1), at(2), at(3), at(4), at(5), 1, 128, far, far, far, far, far, far, 1e-6, 1, 3)
    gemm = fp8._GEMM.pack(at(0), at(1), at(2), at(3), at(4), 1, 128, 128, far, 128, far, far, far, far, far, 4, 4, 1, 0, 0)
    for fn, call in (("quant_fp8", quant), ("rms_norm_fp8", norm), ("gemm_fp8", gemm)):
        assert getattr(sdt.lib(), fn)(call, None) == -4, (fn, sdt.lib().sdt_last_error())  # past every check: no GPU
