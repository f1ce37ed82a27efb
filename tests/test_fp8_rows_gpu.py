"""quant_fp8 and rms_norm_fp8 against 64 bits: widths, types, strides, zeros, infinities and NaN."""
import math

import pytest
import torch

import shape_driven_tile_gb300 as sdt
from _fp8 import E4M3, assert_near, assert_quantised, numbers

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]
WIDTHS = [8, 56, 64, 72, 128, 136, 248, 256, 264, 1000, 4096, 4104, 8192, 8200, 16384, 16392, 32768]


def rows(t, d, dtype, seed, device="cuda", scale=1.0):
    g = torch.Generator(device=device).manual_seed(seed)
    return (scale * torch.randn((t, d), generator=g, device=device)).to(dtype)


def act64(kind, g):
    g = g.double()
    return g * torch.sigmoid(g if kind == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))


# fp32 arithmetic of an activation, per value: the exponential is off by at most 2^-22 and half a step
# of each argument's size times it (arguments up to 30 here: 30 * 2^-22 covers the rounding of a product
# in front of it), the sum, quotient and products by a few half steps
ACT_SLACK = 34 * 2.0 ** -22


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", WIDTHS + [65536])
def test_quant(cuda_device, width, dtype):
    for t in (1, 3, 17):
        x = rows(t, width, dtype, width + t)
        q, s = sdt.quant_fp8(x)
        assert q.dtype is E4M3 and q.shape == x.shape and s.shape == (t, -(-width // 128))
        assert_quantised(q, s, x.double(), 0.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("t,width", [(1, 8), (5, 136), (16, 4096), (333, 1000), (2, 65536)])
def test_gated(cuda_device, t, width, kind, dtype):
    both = rows(t, 2 * width, dtype, t + width, scale=2.0)
    gate, up = both[:, :width], both[:, width:]
    q, s = sdt.quant_fp8(up, gate, activation=kind)
    assert_quantised(q, s, act64(kind, gate) * up.double(), ACT_SLACK)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gates_at_the_ends_of_the_range(cuda_device, kind):
    gate = torch.zeros((2, 128), dtype=torch.bfloat16, device=cuda_device)
    gate[0, 0], gate[0, 1], gate[1, 0] = 3e38, -3e38, -200.0
    up = torch.ones_like(gate)
    q, s = sdt.quant_fp8(up, gate, activation=kind)
    n = numbers(q, s)
    assert n.isfinite().all() and n[0, 1] == 0 and abs(n[0, 0].item() / 3e38 - 1) < 2.0 ** -4
    assert (n[1].abs() < 1e-30).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("width", WIDTHS)
def test_norm(cuda_device, width, residual, dtype):
    for t in (1, 5, 130):
        x, w = rows(t, width, dtype, width + t), rows(1, width, dtype, 7)[0]
        r = rows(t, width, dtype, 8, scale=4.0) if residual else None
        want_r = (x.float() + r.float()).to(dtype) if residual else x
        out = torch.empty_like(x)
        q, s = sdt.rms_norm_fp8(x, w, r, eps=1e-5, out=out)
        if residual:
            assert torch.equal(r, want_r)
        v = want_r.double()
        y = v * w.double() / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-5)
        # a sum of `width` squares in fp32, its root (rsqrt is good to 2 steps), two products
        slack = (width / 8 + 8 + 8) * 2.0 ** -24
        assert_quantised(q, s, y, slack)
        assert_near(out, y, slack * y.abs())


@pytest.mark.parametrize("width", [64, 4096, 16392])
def test_norm_with_a_wide_weight(cuda_device, width):
    x, w = rows(9, width, torch.bfloat16, 3), rows(1, width, torch.float32, 4)[0]
    q, s = sdt.rms_norm_fp8(x, w)
    v = x.double()
    assert_quantised(q, s, v * w.double() / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6), (width / 8 + 16) * 2.0 ** -24)


def test_strides(cuda_device):
    """Slices of wider rows, scales of either order, outputs of the caller's."""
    with pytest.raises(sdt.SdtError, match="row stride of x"):
        sdt.quant_fp8(rows(37, 700, torch.float16, 5)[:, 8:400])
    both = rows(37, 704, torch.float16, 5)
    x, w = both[:, 8:400], torch.ones(392, dtype=torch.float16, device=cuda_device)
    qs = torch.zeros((37, 408), device=cuda_device).to(E4M3)
    scales = torch.zeros((4, 37), device=cuda_device).t()
    want_q, want_s = sdt.quant_fp8(x.contiguous())
    got = sdt.quant_fp8(x, q=qs[:, 8:400], scales=scales)
    assert got[1] is scales and torch.equal(scales, want_s) and torch.equal(qs[:, 8:400].float(), want_q.float())
    assert (qs[:, :8].float() == 0).all() and (qs[:, 400:].float() == 0).all()
    res = rows(37, 800, torch.float16, 6)
    kept = res.clone()
    plain = kept[:, 16:408].contiguous()
    want_q, want_s = sdt.rms_norm_fp8(x.contiguous(), w, plain)
    q, s = sdt.rms_norm_fp8(x, w, res[:, 16:408], scales=scales)
    assert torch.equal(q.float(), want_q.float()) and torch.equal(s, want_s) and torch.equal(res[:, 16:408], plain)
    assert torch.equal(res[:, :16], kept[:, :16]) and torch.equal(res[:, 408:], kept[:, 408:])
    one = x[:1].expand(5, 392)  # one row for every token
    assert torch.equal(sdt.quant_fp8(one)[0].float(), sdt.quant_fp8(one.contiguous())[0].float())


@pytest.mark.parametrize("dtype", TYPES)
def test_zeros_and_tiny_values(cuda_device, dtype):
    x = torch.zeros((3, 264), dtype=dtype, device=cuda_device)
    x[1, 130] = torch.finfo(dtype).smallest_normal
    x[2, 0] = torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    q, s = sdt.quant_fp8(x)
    assert_quantised(q, s, x.double(), 0.0)
    q, s = sdt.rms_norm_fp8(x, torch.ones(264, dtype=dtype, device=cuda_device), eps=1e-6)
    assert (numbers(q, s)[0] == 0).all() and numbers(q, s).isfinite().all()


@pytest.mark.parametrize("dtype", TYPES)
def test_nan_and_infinity_stay_in_their_blocks(cuda_device, dtype):
    x = rows(4, 392, dtype, 9)
    clean_q, clean_s = sdt.quant_fp8(x)
    clean = numbers(clean_q, clean_s)
    x[1, 5], x[2, 200] = torch.nan, -torch.inf
    q, s = sdt.quant_fp8(x)
    n = numbers(q, s)
    assert n[1, 5].isnan() and n[2, 128:256].isnan().all()
    assert torch.equal(n[1, 128:], clean[1, 128:]) and torch.equal(n[2, :128], clean[2, :128]) and torch.equal(n[2, 256:], clean[2, 256:])
    assert torch.equal(n[0], clean[0]) and torch.equal(n[3], clean[3]) and n[1, :5].isfinite().all()
    n = numbers(*sdt.rms_norm_fp8(x, torch.ones(392, dtype=dtype, device=cuda_device)))
    assert n[1].isnan().all() and n[0].isfinite().all() and n[3].isfinite().all()
    assert not (n[2].isfinite() & (n[2] != 0)).any()  # an infinite mean: zeros, and NaN in the infinity's block


@pytest.mark.parametrize("dtype", TYPES)
def test_the_largest_values(cuda_device, dtype):
    top = torch.finfo(dtype).max
    x = torch.full((2, 128), top, dtype=dtype, device=cuda_device)
    x[1, ::2] = -top
    q, s = sdt.quant_fp8(x)
    assert (q.float().abs() == 448).all() and torch.allclose(numbers(q, s), x.double(), rtol=2.0 ** -22)


def test_captured_and_on_another_stream(cuda_device):
    x, r = rows(40, 4096, torch.bfloat16, 11), rows(40, 4096, torch.bfloat16, 12)
    w = torch.ones(4096, dtype=torch.bfloat16, device=cuda_device)
    kept = r.clone()
    want = [t.float() for t in sdt.rms_norm_fp8(x, w, r)] + [t.float() for t in sdt.quant_fp8(x, kept)]
    other = torch.cuda.Stream()
    r.copy_(kept)
    other.wait_stream(torch.cuda.current_stream())
    got = [*sdt.rms_norm_fp8(x, w, r, stream=other), *sdt.quant_fp8(x, kept, stream=other)]
    torch.cuda.current_stream().wait_stream(other)
    assert all(torch.equal(a.float(), b) for a, b in zip(got, want))
    r.copy_(kept)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [*sdt.rms_norm_fp8(x, w, r), *sdt.quant_fp8(x, kept)]
    for _ in range(2):
        r.copy_(kept)
        graph.replay()
        assert all(torch.equal(a.float(), b) for a, b in zip(got, want))


def test_one_row_does_not_depend_on_others(cuda_device):
    """A row alone and among others: the same bits quantised; normed, the same values (the order of a row's sum
    depends on the number of rows)."""
    x = rows(700, 2048, torch.bfloat16, 13)
    w = rows(1, 2048, torch.bfloat16, 14)[0]
    all_q, all_s = sdt.quant_fp8(x)
    q, s = sdt.quant_fp8(x[300:301])
    assert torch.equal(q.float(), all_q[300:301].float()) and torch.equal(s, all_s[300:301])
    v = x[300:301].double()
    y = v * w.double() / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6)
    for q, s in (sdt.rms_norm_fp8(x[300:301], w), [t[300:301] for t in sdt.rms_norm_fp8(x, w)]):
        assert_quantised(q, s, y, (2048 / 8 + 16) * 2.0 ** -24)


def test_rows_past_32_bits(cuda_device):
    """Inputs of more than 2^32 bytes: the last rows are those of a call on them alone."""
    t, d = 270000, 8192
    x = torch.zeros((t, d), dtype=torch.bfloat16, device=cuda_device)
    tail = rows(3, d, torch.bfloat16, 15)
    x[-3:] = tail
    w = rows(1, d, torch.bfloat16, 16)[0]
    q, s = sdt.quant_fp8(x)
    want = sdt.quant_fp8(tail)
    assert torch.equal(q[-3:].float(), want[0].float()) and torch.equal(s[-3:], want[1]) and (q[-4].float() == 0).all()
    q, s = sdt.rms_norm_fp8(x, w, x.clone(), q=q, scales=s)
    v = (tail.float() + tail.float()).to(torch.bfloat16).double()
    y = v * w.double() / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6)
    assert_quantised(q[-3:], s[-3:], y, (d / 8 + 16) * 2.0 ** -24)
    del x, q, s
    torch.cuda.empty_cache()
