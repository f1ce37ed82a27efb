"""Plain 64-bit forms of the 8-bit layer's operators, and the error that fp32 sums may have."""
import torch

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}  # half a step of subnormals


def fp8_values(shape, seed, dtype=E4M3, device="cuda"):
    top = 448.0 if dtype is E4M3 else 57344.0
    g = torch.Generator(device=device).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=device) * (top / 3)).clamp_(-top, top).to(dtype)


def scale_values(shape, seed, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    return torch.empty(shape, device=device).uniform_(1e-3, 3e-3, generator=g)


def numbers(q, scales, rows=1):
    """What fp8 values and their scales stand for, in 64 bits."""
    s = scales.double().repeat_interleave(rows, 0)[: q.shape[0]].repeat_interleave(128, 1)[:, : q.shape[1]]
    return q.double() * s


def product(a, sa, w, sw):
    """(the product in 64 bits, the error that the kernels' fp32 arithmetic may have).

    A block's 128 products are exact and added one after another at worst, each sum off by a
    step (2^-23, the tensor cores may cut instead of rounding); the product of the scales, its
    product with the block sum and each sum over blocks are off by half a step."""
    x, y = numbers(a, sa), numbers(w, sw, 128)
    blocks = -(-a.shape[1] // 128)
    return x @ y.t(), (128 * 2.0 ** -23 + (blocks + 2) * 2.0 ** -24) * (x.abs() @ y.abs().t())


def assert_near(got, want, slack, dtype=None):
    """got is want rounded to its type, but for `slack` before the rounding."""
    dtype = dtype or got.dtype
    off = (got.double() - want).abs()
    allowed = slack + STEP[dtype] * (want.abs() + slack) + TINY[dtype]
    bad = ~(off <= allowed)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, by up to {float((off / allowed).max()):.3g} of what is allowed"


def e4m3_grid(v):
    """Nearest e4m3 numbers of 64-bit values of at most 448, ties to even."""
    step = torch.exp2(torch.frexp(v)[1].double().sub(1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def assert_quantised(q, scales, y, slack):
    """q and scales are those of the 64-bit rows y, known up to a relative `slack` (of each value)."""
    tokens, width = y.shape
    blocks = torch.nn.functional.pad(y, (0, -width % 128)).unflatten(1, (-1, 128))
    top = blocks.abs().amax(2).clamp(min=2.0 ** -100)
    want = top / 448
    assert ((scales.double() - want).abs() <= (slack + 3 * 2.0 ** -24) * want).all()
    # before its rounding a value is off by slack, the quotient 448 / top and a product (and top's own slack)
    ratio = (blocks / want.unsqueeze(2)).flatten(1)[:, :width]
    moved = ratio * (2 * slack + 4 * 2.0 ** -24)
    lo, hi = (e4m3_grid((ratio + s * moved.abs()).clamp(-448, 448)) for s in (-1, 1))
    got = q.double()
    bad = (got < lo) | (got > hi)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} values are not the nearest"
