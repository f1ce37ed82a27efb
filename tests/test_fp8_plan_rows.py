"""gemm_fp8's choice of tile goes by where rows start, not by the number of values in them (no GPU needed)."""
import ctypes

import pytest

import shape_driven_tile_gb300 as sdt
from shape_driven_tile_gb300 import fp8

NULL, SHAPE, ARG = -1, -3, -10
A = 0x10000


def plan(m, n, k, lda, ldw, a=A, w=A, tile=0, splits=0, sms=152):
    kb = -(-k // 128)
    out = ctypes.c_int(), ctypes.c_int()
    call = fp8._GEMM.pack(a, A, w, A, 1 << 50, m, n, k, lda, ldw, n, kb, 1, kb, 1, 4, 4, 1, tile, splits)
    rc = sdt.lib().sdt_gemm_fp8_plan_call(call, sms, *(ctypes.byref(x) for x in out))
    return rc if rc else tuple(x.value for x in out)


# (k, a's rows, w's rows, a's base, w's base): measured with tiles of 128 and 192, 333 tokens, 5000 outputs
@pytest.mark.parametrize("k,lda,ldw,a,w,tile", [
    (4208, 4208, 4208, 0, 0, 192),    # 16.8 and 15.5 us
    (4208, 4224, 4224, 0, 0, 128),    # 13.7, 14.9
    (4208, 4208, 4224, 0, 0, 128),    # 14.4, 15.2
    (4208, 4224, 4208, 0, 0, 128),    # 14.2, 15.1
    (4208, 4224, 4224, 16, 16, 192),  # 18.2, 16.7
    (4224, 4224, 4224, 0, 0, 128),    # 13.7, 14.9
    (4224, 4240, 4240, 0, 0, 192),    # 16.7, 15.6
    (4224, 4240, 4224, 0, 0, 128),    # 14.3, 15.1
    (4224, 4224, 4224, 16, 16, 192),  # 18.2, 16.7
])
def test_where_rows_start(k, lda, ldw, a, w, tile):
    assert plan(333, 5000, k, lda, ldw, A + a, A + w) == (tile, 1)


def test_the_binding_and_the_sizes_alone():
    assert sdt.gemm_fp8_plan(333, 5000, 4208) == (192, 1) == sdt.gemm_fp8_plan(333, 5000, 4208, lda=4208, ldw=4208)
    assert sdt.gemm_fp8_plan(333, 5000, 4208, lda=4224, ldw=4224) == (128, 1) == sdt.gemm_fp8_plan(333, 5000, 4208, lda=4224)
    assert sdt.gemm_fp8_plan(333, 5000, 4216) == (128, 1)  # rows of 4216 are 4224 apart
    for m, n, k in ((1, 12288, 4096), (48, 4096, 14336), (4096, 4096, 4096)):
        assert sdt.gemm_fp8_plan(m, n, k) == sdt.gemm_fp8_plan(m, n, k, lda=k) == plan(m, n, k, k, k)


def test_what_the_call_asks_for():
    assert plan(333, 5000, 4208, 4208, 4208, tile=64, splits=3) == (64, 3)
    assert plan(333, 5000, 200, 208, 208, tile=16, splits=8) == (16, 2)  # no more than blocks
    assert plan(333, 5000, 4208, 4208, 4208, tile=256, splits=3) == (256, 1)


def test_refusals():
    assert plan(0, 64, 64, 64, 64) == SHAPE and plan(4, 64, 0, 64, 64) == SHAPE and plan(4, 64, 64, 64, 64, sms=0) == SHAPE
    assert plan(4, 64, 64, 72, 64) == ARG
    assert sdt.lib().sdt_gemm_fp8_plan_call(None, 152, None, None) == NULL
    with pytest.raises(sdt.SdtError):
        sdt.gemm_fp8_plan(333, 5000, 4208, lda=4200)
