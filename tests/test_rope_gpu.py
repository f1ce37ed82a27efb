"""rope_qk against rotations in 64 bits: layouts, parts of heads, strides, far positions, in place."""
import math

import numpy as np
import pytest
import torch

import shape_driven_tile_gb300 as sdt
from _fp8 import assert_near

pytestmark = pytest.mark.gpu


def turned(x, positions, table, inverse=False):
    """(the rotation in 64 bits, what fp32 arithmetic may be off before the rounding)."""
    half = table.rotary // 2
    first = torch.arange(half, device=x.device) * (2 if table.interleaved else 1)
    second = first + 1 if table.interleaved else first + half
    # extended precision on the host: 64-bit angles of far positions are off by 2^-53 of them
    angle = np.multiply.outer(positions.cpu().numpy().astype(np.longdouble), np.array(table.frequencies, dtype=np.longdouble))
    cos, sin = (torch.from_numpy((f(angle) * table.magnitude).astype(np.float64)).to(x.device)[:, None] for f in (np.cos, np.sin))
    if inverse:
        sin = -sin
    a, b, y = x[..., first].double(), x[..., second].double(), x.double()
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    # the angle is off by 2^-25 turns, sine and cosine by 2 steps, then two products and a sum
    slack = torch.zeros_like(y)
    slack[..., first] = slack[..., second] = (2 * math.pi * 2.0 ** -25 + 8 * 2.0 ** -24) * abs(table.magnitude) * (a.abs() + b.abs())
    return y, slack


def inputs(t, hq, hk, d, dtype, seed=0, longest=5000, pos=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k = (torch.randn((t, h, d), generator=g, device="cuda").to(dtype) for h in (hq, hk))
    return q, k, torch.randint(0, longest, (t,), generator=g, device="cuda").to(pos)


def check(q, k, positions, table, inverse=False, **kw):
    want = [turned(x, positions, table, inverse) for x in (q, k)]
    got = sdt.rope_qk(q, k, positions, table, inverse=inverse, **kw)
    for o, (y, slack) in zip(got, want):
        assert_near(o, y, slack)
        assert torch.equal(o[..., table.rotary:].double(), y[..., table.rotary:])
    return got


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rotary", [(128, 128), (128, 96), (64, 64), (80, 40), (80, 20), (256, 64), (96, 96), (6, 2), (40, 36), (2, 2), (72, 14)])
def test_layouts(cuda_device, d, rotary, interleaved, dtype):
    table = sdt.RopeTable(rotary, interleaved=interleaved)
    for t, hq, hk in ((1, 1, 1), (7, 5, 3), (130, 8, 2)):
        q, k, pos = inputs(t, hq, hk, d, dtype, seed=t)
        check(q, k, pos, table)
        check(q, k, pos, table, inverse=True)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [128, 64, 20])
def test_in_place_in_the_rows_of_a_projection(cuda_device, rotary, interleaved):
    table = sdt.RopeTable(rotary, interleaved=interleaved)
    rows = torch.randn((33, 12 * 128 + 8), device=cuda_device).to(torch.bfloat16)
    kept = rows.clone()
    q, k = rows[:, :8 * 128].unflatten(1, (8, 128)), rows[:, 8 * 128:10 * 128].unflatten(1, (2, 128))
    pos = torch.arange(33, device=cuda_device, dtype=torch.int32) * 77
    want = [turned(x, pos, table) for x in (q, k)]
    got = sdt.rope_qk(q, k, pos, table, q_out=q, k_out=k)
    assert got[0] is q and got[1] is k
    for o, (y, slack) in zip(got, want):
        assert_near(o, y, slack)
    assert torch.equal(rows[:, 10 * 128:], kept[:, 10 * 128:])


@pytest.mark.parametrize("shift", [0, 1, 2, 4])
def test_any_strides_and_alignment(cuda_device, shift):
    """Heads outside tokens, odd rows, bases of two bytes."""
    table = sdt.RopeTable(64)
    base = torch.randn(4 * 50 * 130 + 8, device=cuda_device).to(torch.float16)
    q = base[shift:shift + 4 * 50 * 130].view(4, 50, 130)[..., :128].transpose(0, 1)
    k = base[shift:shift + 50 * 260].view(50, 260)[:, 3:131].unsqueeze(1)
    pos = torch.arange(50, device=cuda_device)
    check(q, k, pos, table)
    out = torch.empty((4, 50, 128), dtype=torch.float16, device=cuda_device).transpose(0, 1)
    check(q, k, pos, table, q_out=out)
    check(q[:1].expand(50, 4, 128), k, pos, table)  # one token's queries for every position


@pytest.mark.parametrize("scaling,kw", [("none", {}), ("linear", dict(factor=8.0)), ("base", dict(factor=4.0)),
                                        ("ramp", dict(factor=40.0, original_length=4096)),
                                        ("smooth", dict(factor=8.0, original_length=8192, base=500000.0))])
def test_far_positions(cuda_device, scaling, kw):
    table = sdt.RopeTable(128, scaling=scaling, **kw)
    q, k, _ = inputs(9, 4, 1, 128, torch.float16, seed=2)
    pos = torch.tensor([0, 1, 4095, 131071, 1048575, 16777217, 2 ** 31 - 1, -1, -70000], device=cuda_device)
    check(q, k, pos, table)
    check(q, k, pos.to(torch.int32), table)


def test_queries_alone_and_no_heads(cuda_device):
    table = sdt.RopeTable(64)
    q, k, pos = inputs(11, 3, 1, 64, torch.bfloat16)
    both = sdt.rope_qk(q, k, pos, table)
    one = sdt.rope_qk(q, None, pos, table)
    assert one[1] is None and torch.equal(one[0], both[0])
    none = sdt.rope_qk(q[:, :0], k, pos, table)
    assert none[0].shape == (11, 0, 64) and torch.equal(none[1], both[1])
    assert sdt.rope_qk(q[:0], k[:0], pos[:0], table)[0].shape == (0, 3, 64)


def test_own_frequencies_and_magnitude(cuda_device):
    table = sdt.RopeTable(6, frequencies=[7.0, 0.0, -0.25], magnitude=-1.5)
    q, k, pos = inputs(20, 2, 2, 8, torch.float16, seed=4)
    check(q, k, pos, table)


def test_inverse_is_the_transpose(cuda_device):
    """Gradients: <rope(x), g> = <x, rope(g, inverse)>, and differences of outputs are outputs of differences."""
    table = sdt.RopeTable(64, scaling="ramp", factor=4.0, original_length=1024)
    x, g, pos = inputs(64, 4, 4, 64, torch.float16, seed=5)
    y = sdt.rope_qk(x, None, pos, table)[0]
    back = sdt.rope_qk(g, None, pos, table, inverse=True)[0]
    want, _ = turned(g, pos, table, inverse=True)
    a, b, c = (y.double() * g.double()).sum(), (x.double() * back.double()).sum(), (x.double() * want).sum()
    # each of the 2 * 64 * 4 * 64 rounded values is off by at most 2^-11 of itself
    room = 2.0 ** -11 * ((y.double() * g.double()).abs().sum() + (x.double() * back.double()).abs().sum()) * 1.01
    assert abs(a - b) <= room and abs(b - c) <= room


def test_infinities_and_nan_stay_in_their_pairs(cuda_device):
    table = sdt.RopeTable(128)
    q, k, pos = inputs(5, 2, 1, 128, torch.bfloat16, seed=6)
    clean = sdt.rope_qk(q, k, pos, table)
    q[2, 1, 10], k[3, 0, 127] = torch.nan, torch.inf
    got = sdt.rope_qk(q, k, pos, table)
    hit = torch.zeros_like(q, dtype=torch.bool)
    hit[2, 1, [10, 74]] = True
    assert got[0][hit].isnan().all() and torch.equal(got[0][~hit], clean[0][~hit])
    hit = torch.zeros_like(k, dtype=torch.bool)
    hit[3, 0, [63, 127]] = True
    assert not got[1][hit].isfinite().any() and torch.equal(got[1][~hit], clean[1][~hit])


def test_captured_and_on_another_stream(cuda_device):
    table = sdt.RopeTable(128)
    q, k, pos = inputs(64, 8, 2, 128, torch.bfloat16, seed=7)
    want = sdt.rope_qk(q, k, pos, table)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = sdt.rope_qk(q, k, pos, table, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sdt.rope_qk(q, k, pos, table)
    pos.add_(3)
    graph.replay()
    want = sdt.rope_qk(q, k, pos, table)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
