"""Outputs in the rows that hold the inputs, beside them: what the host takes, the kernels compute as in tensors of their own."""
import pytest
import torch

import shape_driven_tile_gb300 as sdt
from _fp8 import E4M3, fp8_values, scale_values

pytestmark = pytest.mark.gpu


def part(rows, lo, hi, dtype):
    """Bytes lo .. hi of each row as `dtype`."""
    return rows[:, lo:hi].view(dtype)


def test_rows_of_everything(cuda_device):
    """x, residual, 16-bit output, fp8 values and scales side by side."""
    t, d, g = 700, 640, torch.Generator(device=cuda_device).manual_seed(1)
    wide = 2 * d  # bytes of a row in 16 bits
    rows = torch.zeros((t, 3 * wide + d + 5 * 4 + 12), dtype=torch.uint8, device=cuda_device)
    x, r, out = (part(rows, i * wide, (i + 1) * wide, torch.bfloat16) for i in range(3))
    q, s = part(rows, 3 * wide, 3 * wide + d, E4M3), part(rows, 3 * wide + d, 3 * wide + d + 5 * 4, torch.float32)
    x.copy_(torch.randn((t, d), generator=g, device=cuda_device))
    r.copy_(torch.randn((t, d), generator=g, device=cuda_device))
    w, r1, out1 = torch.ones(d, dtype=torch.bfloat16, device=cuda_device), r.clone(), torch.empty((t, d), dtype=torch.bfloat16, device=cuda_device)
    q1, s1 = sdt.rms_norm_fp8(x.clone(), w, r1, out=out1)
    kept = x.clone()
    sdt.rms_norm_fp8(x, w, r, out=out, q=q, scales=s)
    for a, b in ((x, kept), (r, r1), (out, out1), (s, s1), (q.view(torch.uint8), q1.view(torch.uint8))):
        assert torch.equal(a, b)
    assert (rows[:, 3 * wide + d + 5 * 4:] == 0).all()
    q1, s1 = sdt.quant_fp8(x.clone(), r.clone())
    sdt.quant_fp8(x, r, q=q, scales=s)
    assert torch.equal(q.view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s, s1)
    with pytest.raises(sdt.SdtError, match="overlap"):
        sdt.rms_norm_fp8(x, w, r, out=r)
    with pytest.raises(sdt.SdtError, match="overlap"):
        sdt.rms_norm_fp8(x, w, x)
    with pytest.raises(sdt.SdtError, match="overlap"):
        sdt.quant_fp8(x, q=part(rows, d, 2 * d, E4M3))


@pytest.mark.parametrize("m", [3, 300])
def test_a_product_beside_its_operand(cuda_device, m):
    n, k = 256, 384
    rows = torch.zeros((m, 384 + 512), dtype=torch.uint8, device=cuda_device)
    a, c = part(rows, 0, 384, E4M3), part(rows, 384, 896, torch.bfloat16)
    a.view(torch.uint8).copy_(fp8_values((m, k), 1).view(torch.uint8))
    sa, w, sw = scale_values((m, 3), 2), fp8_values((n, k), 3), scale_values((2, 3), 4)
    want = sdt.gemm_fp8(a.clone(), sa, w, sw)
    sdt.gemm_fp8(a, sa, w, sw, c)
    assert torch.equal(c, want)
    with pytest.raises(sdt.SdtError, match="overlap"):
        sdt.gemm_fp8(a, sa, w, sw, part(rows, 368, 880, torch.bfloat16))


def test_turned_into_other_slices_of_the_rows(cuda_device):
    table, pos = sdt.RopeTable(64), torch.arange(50, device=cuda_device)
    rows = torch.randn((50, 2 * (4 + 2) * 64), device=cuda_device).to(torch.bfloat16)
    q, k, qo, ko = (t.unflatten(1, (-1, 64)) for t in rows.split((256, 128, 256, 128), 1))
    want = sdt.rope_qk(q.clone(), k.clone(), pos, table)
    got = sdt.rope_qk(q, k, pos, table, q_out=qo, k_out=ko)
    assert got[0] is qo and got[1] is ko and torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    with pytest.raises(sdt.SdtError, match="overlap"):
        sdt.rope_qk(q, k, pos, table, q_out=rows[:, 384:640].unflatten(1, (-1, 64)), k_out=rows[:, 512:640].unflatten(1, (-1, 64)))
