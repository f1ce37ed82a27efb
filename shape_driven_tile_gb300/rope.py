"""Rotary positions of queries and keys, before the keys go into the cache.

``RopeTable`` holds the frequencies of a model's positions; ``rope_qk`` checks and marshals
arguments and calls the C entry point of the same name (include/sdt.h).
"""
from __future__ import annotations

import math
import struct

import torch

from . import _streams
from ._lib import check
from .fp8 import _current_device, _current_stream, _fn

VALUE_CODES = {torch.float16: 0, torch.bfloat16: 1}
POSITION_BYTES = {torch.int32: 4, torch.int64: 8}
SCALINGS = ("none", "linear", "base", "ramp", "smooth")
# sdt_rope_qk (include/sdt.h)
_ROPE = struct.Struct("6P13qf4i0q")


def rope_frequencies(rotary: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                     original_length: int | None = None, low: float = 1.0, high: float | None = None):
    """(frequencies, magnitude): radians per position of each of the rotary // 2 pairs in double
    precision, and the factor on the rotated values.

    scaling "none": base ** (-2 i / rotary).  For contexts `factor` times as long as the
    original_length that a model was trained on: "linear" divides every frequency by factor;
    "base" takes base * factor ** (rotary / (rotary - 2)); "ramp" and "smooth" keep the
    frequencies that turn more than `high` times over original_length, divide those that turn
    fewer than `low` times, and blend between them: "ramp" (high 32 by default) evenly over the
    pairs, with a magnitude of 0.1 ln(factor) + 1, "smooth" (high 4) evenly over the turns.
    """
    if scaling not in SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(map(repr, SCALINGS))}, got {scaling!r}")
    if not hasattr(rotary, "__index__"):
        raise TypeError(f"rotary must be an integer, got {type(rotary).__name__}")
    if rotary < 2 or rotary % 2:
        raise ValueError(f"rotary must be even and positive, got {rotary}")
    if not (base > 1.0 and math.isfinite(base)):
        raise ValueError(f"base must be a number above 1, got {base}")
    if not (factor >= 1.0 and math.isfinite(factor)):
        raise ValueError(f"factor must be a number of at least 1, got {factor}")
    if scaling == "base":
        if rotary < 4:
            raise ValueError("scaling 'base' needs rotary of at least 4")
        base = base * factor ** (rotary / (rotary - 2))
    freq = [base ** (-2.0 * i / rotary) for i in range(rotary // 2)]
    if scaling == "linear":
        freq = [f / factor for f in freq]
    if scaling in ("none", "linear", "base"):
        return freq, 1.0
    if high is None:
        high = 32.0 if scaling == "ramp" else 4.0
    if original_length is None or original_length < 1:
        raise ValueError(f"scaling {scaling!r} needs original_length")
    if not 0.0 < low < high:
        raise ValueError(f"low and high must be positive, low below high, got {low} and {high}")

    def pair_that_turns(times):
        return rotary * math.log(original_length / (times * 2.0 * math.pi)) / (2.0 * math.log(base))

    first = max(0, math.floor(pair_that_turns(high)))
    last = min(rotary - 1, math.ceil(pair_that_turns(low)))
    scaled = []
    for i, f in enumerate(freq):
        if scaling == "ramp":
            divided = (i - first) / max(last - first, 1e-3)
        else:
            divided = (high - original_length * f / (2.0 * math.pi)) / (high - low)
        divided = min(1.0, max(0.0, divided))
        scaled.append(f * (1.0 - divided) + f / factor * divided)
    return scaled, 0.1 * math.log(factor) + 1.0 if scaling == "ramp" else 1.0


class RopeTable:
    """The frequencies of a model's rotary positions, on the GPU.

    rotary: how many of a head's first values are rotated (even).  interleaved: pairs are
    (2 i, 2 i + 1) instead of (i, rotary // 2 + i).  The rest as rope_frequencies; or
    ``frequencies`` (radians per position, rotary // 2 numbers) and ``magnitude`` of one's own.
    They are kept as 64-bit fractions of a turn, so that any position turns exactly.
    """

    def __init__(self, rotary: int, base: float = 10000.0, *, interleaved: bool = False, scaling: str = "none", factor: float = 1.0,
                 original_length: int | None = None, low: float = 1.0, high: float | None = None, frequencies=None,
                 magnitude: float | None = None, device=None):
        if frequencies is None:
            frequencies, own = rope_frequencies(rotary, base, scaling=scaling, factor=factor, original_length=original_length,
                                                low=low, high=high)
        else:
            if not hasattr(rotary, "__index__"):
                raise TypeError(f"rotary must be an integer, got {type(rotary).__name__}")
            frequencies, own = [float(f) for f in frequencies], 1.0
            if rotary != 2 * len(frequencies) or not frequencies:
                raise ValueError(f"frequencies must be rotary // 2 = {rotary // 2} numbers, got {len(frequencies)}")
        if not all(math.isfinite(f) for f in frequencies):
            raise ValueError("frequencies must be finite")
        self.rotary, self.interleaved = rotary, bool(interleaved)
        self.magnitude = own if magnitude is None else float(magnitude)
        if not math.isfinite(self.magnitude) or abs(self.magnitude) > 1e30:
            raise ValueError(f"magnitude is out of range: {magnitude}")
        self.frequencies = tuple(frequencies)
        turns = [_turns(f) for f in frequencies]
        self.turns = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=device or "cuda")
        self.turns_ptr, self.device_index = self.turns.data_ptr(), self.turns.get_device()


def _turns(frequency: float) -> int:
    """frequency / (2 pi) modulo 1 as a fraction of 2^64 (the double's own 53 bits, divided in more)."""
    mantissa, exponent = math.frexp(frequency)
    top = int(mantissa * (1 << 53))  # frequency = top * 2^(exponent - 53)
    shift = exponent - 53 + 64 + 128
    scaled = top << shift if shift >= 0 else top >> -shift  # frequency * 2^192
    # 2 pi * 2^128, to the nearest integer
    return (scaled // 2138057168129933495719360746323741566601) % (1 << 64)


def _need(t, name, dtypes, dims):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must be {dims}-D")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != _current_device():
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{_current_device()}")


def _need_heads(t, name, dtypes, shape):
    _need(t, name, dtypes, 3)
    if any(want is not None and have != want for have, want in zip(t.shape, shape)):
        raise ValueError(f"{name} must be {tuple('any' if w is None else w for w in shape)}, got {tuple(t.shape)}")
    if t.stride(2) != 1 and t.shape[2] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def rope_qk(q, k, positions, table: RopeTable, *, q_out=None, k_out=None, inverse: bool = False, stream=None):
    """Queries and keys turned to their positions; returns (q_out, k_out).

    q: [tokens, q_heads, head_dim], k: [tokens, k_heads, head_dim] or None, float16 or bfloat16,
    any strides with head_dim contiguous (slices of a fused projection's rows may be given).
    positions: int32 or int64 [tokens].  With (x, y) a pair of a head and t = position *
    frequency: (x cos t - y sin t, y cos t + x sin t) * magnitude, in float32, rounded once;
    values from table.rotary on are copied.  q_out, k_out: q and k themselves to work in place,
    or tensors apart from both; new ones if None.  inverse: turns back (gradients of the outputs
    to gradients of the inputs).
    """
    try:
        dev, dtype = _current_device(), q.dtype
        tokens, q_heads, head_dim = q.shape
        q_token, q_head, along = q.stride()
        k_heads = k_ptr = k_token = k_head = 0
        good = (table.device_index == dev and table.rotary <= head_dim and dtype in VALUE_CODES and q.get_device() == dev
                and along == 1 and positions.get_device() == dev and positions.shape == (tokens,)
                and positions.dtype in POSITION_BYTES and positions.is_contiguous())
        if k is not None:
            k_tokens, k_heads, k_dim = k.shape
            k_token, k_head, along = k.stride()
            k_ptr = k.data_ptr()
            good = good and k.dtype is dtype and k_tokens == tokens and k_dim == head_dim and along == 1 and k.get_device() == dev
    except (AttributeError, TypeError, ValueError, RuntimeError):
        good = False
    if not good:
        _need_heads(q, "q", VALUE_CODES, (None, None, None))
        tokens, q_heads, head_dim = q.shape
        if k is not None:
            _need_heads(k, "k", (q.dtype,), (tokens, None, head_dim))
        if not isinstance(table, RopeTable):
            raise TypeError("table must be a RopeTable")
        if table.device_index != _current_device():
            raise ValueError(f"the table is on cuda:{table.device_index}, but the current device is cuda:{_current_device()}")
        if table.rotary > head_dim:
            raise ValueError(f"the table rotates {table.rotary} values of a head, which has {head_dim}")
        _need(positions, "positions", POSITION_BYTES, 1)
        if positions.shape[0] != tokens or not positions.is_contiguous():
            raise ValueError(f"positions must be {tokens} contiguous entries")
    if q_out is q:
        qo_token, qo_head = q_token, q_head
    elif q_out is None:
        q_out = _new(q, stream)
        qo_token, qo_head = q_heads * head_dim, head_dim
    else:
        _need_heads(q_out, "q_out", (dtype,), q.shape)
        qo_token, qo_head, _ = q_out.stride()
    ko_ptr = ko_token = ko_head = 0
    if k is None:
        if k_out is not None:
            raise ValueError("k_out goes with k")
    else:
        if k_out is k:
            ko_token, ko_head = k_token, k_head
        elif k_out is None:
            k_out = _new(k, stream)
            ko_token, ko_head = k_heads * head_dim, head_dim
        else:
            _need_heads(k_out, "k_out", (dtype,), k.shape)
            ko_token, ko_head, _ = k_out.stride()
        ko_ptr = k_out.data_ptr()
    call = _ROPE.pack(q.data_ptr(), k_ptr, q_out.data_ptr(), ko_ptr, positions.data_ptr(), table.turns_ptr, tokens, q_heads, k_heads,
                      head_dim, table.rotary, q_token, q_head, k_token, k_head, qo_token, qo_head, ko_token, ko_head, table.magnitude,
                      VALUE_CODES[dtype], POSITION_BYTES[positions.dtype], table.interleaved, bool(inverse))
    check(_fn("rope_qk")(call, _current_stream(dev) if stream is None else _streams.handle(stream)))
    return q_out, k_out


def _new(x, stream):
    """An output as x, contiguous."""
    if stream is None:
        return torch.empty(x.shape, dtype=x.dtype, device=x.device)
    return _streams.empty(x.shape, x.dtype, x.device, stream)
