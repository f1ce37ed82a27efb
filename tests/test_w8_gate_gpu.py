"""The activations of quant_fp8 over the range of gates, seen through the float32 scales."""
import math

import pytest
import torch

import shape_driven_tile_gb300 as sdt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gates_from_far_below_to_far_above(cuda_device, kind):
    """One gate a block, so that its scale is the activation / 448.  In units of 2^-24 of the value: the exponential instruction
    4 (2^-22), its correction, the sum with 1, and the quotient 1.5 together 3.5, two products 2, the scale 2; gelu's argument
    4.5 (a square, two constants, a multiply-add, a product), which count |t| times."""
    top = 86.5 if kind == "silu" else 10.0
    gates = torch.arange(-top, top + 0.25, 0.5, device=cuda_device)
    gates = gates[gates != 0].to(torch.bfloat16)
    up = torch.full((gates.numel(), 128), 2.0 ** 60, dtype=torch.bfloat16, device=cuda_device)
    q, s = sdt.quant_fp8(up, gates[:, None].expand(-1, 128).contiguous(), activation=kind)
    g = gates.double()
    t = g if kind == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    keep = t > -86.6  # (below, the sigmoid leaves fp32's normal numbers)
    want = (2.0 ** 60 * g / (1 + torch.exp(-t)) / 448).abs()
    room = (11.5 + (0.0 if kind == "silu" else 4.5) * t.abs()) * 2.0 ** -24
    off = ((s[:, 0].double() - want).abs() / want)[keep] / room[keep]
    assert keep.sum() > 30 and off.max() <= 1, (gates[keep][off.argmax()].item(), off.max().item())
    assert (q.float()[keep].abs() == 448).all()
