"""Products in 8 bits and what makes their operands: fp8 values with a float32 scale per 128.

``rms_norm_fp8`` and ``quant_fp8`` turn rows of 16-bit activations into fp8 and scales,
``gemm_fp8`` multiplies them with fp8 weights.  As in the package's other calls, the functions
check and marshal arguments and call the C entry points of the same names (include/sdt.h);
every step runs in the library's kernels on the current stream, without a synchronisation.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _streams
from ._lib import check, lib

BLOCK = 128  # values per scale
OUT_CODES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 3}
FP8_CODES = {torch.float8_e4m3fn: 4, torch.float8_e5m2: 5}
ROW_CODES = {torch.float16: 0, torch.bfloat16: 1}
ACTIVATIONS = {"silu": 1, "gelu": 2}

# sdt_gemm_fp8, sdt_quant_fp8 and sdt_rms_norm_fp8 (include/sdt.h; "0q" is C's padding at the end)
_GEMM, _QUANT, _NORM = struct.Struct("5P10q5i0q"), struct.Struct("4P7q2i0q"), struct.Struct("6P8qf2i0q")
_current_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_F32, _E4M3 = torch.float32, torch.float8_e4m3fn
_functions = {}


def _fn(name):
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(lib(), name)
    return f


def _need(t, name, dtypes, shape):
    """A CUDA tensor on the current device; None in `shape` stands for any size."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != len(shape) or any(want is not None and have != want for have, want in zip(t.shape, shape)):
        raise ValueError(f"{name} must be {tuple('any' if w is None else w for w in shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != _current_device():
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{_current_device()}")


def _need_rows(t, name, dtypes, shape):
    _need(t, name, dtypes, shape)
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _integer(name, value):
    if not hasattr(value, "__index__"):
        raise TypeError(f"{name} must be an integer, got {type(value).__name__}")
    if not -2 ** 31 <= value < 2 ** 31:
        raise ValueError(f"{name} is out of range: {value}")
    return value


def gemm_fp8(a, a_scales, w, w_scales, out=None, *, out_dtype=torch.bfloat16, tile: int = 0, splits: int = 0, stream=None):
    """out = A @ W.T of fp8 values with a scale per 128 of k:
    out[m, n] = sum_k a[m, k] * a_scales[m, k // 128] * w[n, k] * w_scales[n // 128, k // 128].

    a: [M, K] and w: [N, K] (K-major, as gemv_m1's W), float8_e4m3fn or float8_e5m2, rows
    contiguous and 16-byte aligned (padding allowed); N a multiple of 8.  a_scales: float32
    [M, ceil(K / 128)], w_scales: float32 [ceil(N / 128), ceil(K / 128)], any strides.  out:
    [M, N] float16, bfloat16 or float32 (out_dtype if the call allocates it), apart from the
    operands and scales.  Sums are held in float32.  tile, splits: 0 picks (include/sdt.h has the others).
    """
    try:
        dev, dtype = _current_device(), out_dtype if out is None else out.dtype
        (M, K), (N, k2) = a.shape, w.shape
        lda, a1 = a.stride()
        ldw, w1 = w.stride()
        as0, as1 = a_scales.stride()
        ws0, ws1 = w_scales.stride()
        blocks = -(-K // BLOCK)
        good = (k2 == K and (a1 == 1 or K <= 1) and (w1 == 1 or K <= 1) and a_scales.dtype is _F32 and w_scales.dtype is _F32
                and a_scales.shape == (M, blocks) and w_scales.shape == (-(-N // BLOCK), blocks)
                and a.get_device() == dev and w.get_device() == dev and a_scales.get_device() == dev
                and w_scales.get_device() == dev and dtype in OUT_CODES and a.dtype in FP8_CODES and w.dtype in FP8_CODES)
    except (AttributeError, TypeError, ValueError, RuntimeError):
        good = False
    if not good:
        _need_rows(a, "a", FP8_CODES, (None, None))
        M, K = a.shape
        _need_rows(w, "w", FP8_CODES, (None, K))
        blocks = -(-K // BLOCK)
        _need(a_scales, "a_scales", (_F32,), (M, blocks))
        _need(w_scales, "w_scales", (_F32,), (-(-w.shape[0] // BLOCK), blocks))
        if out is None and out_dtype not in OUT_CODES:
            raise TypeError(f"out_dtype must be {' or '.join(map(str, OUT_CODES))}, got {out_dtype}")
        _need_rows(out, "out", OUT_CODES, (M, w.shape[0]))
    if out is None:
        out = torch.empty((M, N), dtype=dtype, device=a.device) if stream is None else _streams.empty((M, N), dtype, a.device, stream)
        ldc = N
    else:
        _need_rows(out, "out", OUT_CODES, (M, N))
        ldc = out.stride(0)
    try:
        call = _GEMM.pack(a.data_ptr(), a_scales.data_ptr(), w.data_ptr(), w_scales.data_ptr(), out.data_ptr(), M, N, K, lda, ldw,
                          ldc, as0, as1, ws0, ws1, FP8_CODES[a.dtype], FP8_CODES[w.dtype], OUT_CODES[dtype], tile, splits)
    except (struct.error, TypeError, ValueError, OverflowError):
        _integer("tile", tile)
        _integer("splits", splits)
        raise
    check(_fn("gemm_fp8")(call, _current_stream(dev) if stream is None else _streams.handle(stream)))
    return out


def gemm_fp8_plan(M: int, N: int, K: int, sm_count: int = 152, *, lda: int | None = None, ldw: int | None = None) -> tuple[int, int]:
    """(tile, splits) that gemm_fp8 picks on a GPU with sm_count SMs; no GPU needed.  lda, ldw: elements from row to row of
    a and w (None: K rounded up to 16); tensors start at multiples of 32 bytes here."""
    tile, splits = ctypes.c_int(), ctypes.c_int()
    at = ctypes.byref(tile), ctypes.byref(splits)
    if lda is None and ldw is None:
        check(lib().sdt_gemm_fp8_plan_for(M, N, K, _integer("sm_count", sm_count), *at))
    else:
        row, blocks, p = -(-K // 16) * 16, -(-K // BLOCK), 4096  # (addresses that nothing follows)
        call = _GEMM.pack(p, p, p, p, 1 << 62, M, N, K, row if lda is None else lda, row if ldw is None else ldw, N, blocks, 1, blocks, 1,
                          FP8_CODES[_E4M3], FP8_CODES[_E4M3], OUT_CODES[torch.bfloat16], 0, 0)
        check(lib().sdt_gemm_fp8_plan_call(call, _integer("sm_count", sm_count), *at))
    return tile.value, splits.value


def _outputs(q, scales, tokens, width, device, stream):
    """(q, scales, their strides) of a call that may be given them."""
    blocks = -(-width // BLOCK)
    if q is None:
        shape = (tokens, width)
        q = torch.empty(shape, dtype=_E4M3, device=device) if stream is None else _streams.empty(shape, _E4M3, device, stream)
        q_row = width
    else:
        _need_rows(q, "q", (_E4M3,), (tokens, width))
        q_row = q.stride(0)
    if scales is None:
        shape = (tokens, blocks)
        scales = torch.empty(shape, dtype=_F32, device=device) if stream is None else _streams.empty(shape, _F32, device, stream)
        return q, scales, q_row, blocks, 1
    _need(scales, "scales", (_F32,), (tokens, blocks))
    return q, scales, q_row, *scales.stride()


def quant_fp8(x, gate=None, *, activation: str = "silu", q=None, scales=None, stream=None):
    """fp8 and scales of x, or of act(gate) * x: gemm_fp8's operand after attention and between
    the two products of a gated feed-forward block.

    x, gate: float16 or bfloat16 [tokens, width], rows contiguous (slices of one product's rows
    may be given), width a multiple of 8 up to 65536.  activation: "silu", or "gelu" (the tanh
    form); it counts only with a gate.  Returns (q, scales): float8_e4m3fn [tokens, width] and
    float32 [tokens, ceil(width / 128)] with x = q * scales, where a block's scale is its
    largest absolute value / 448; q and scales may be given (scales with any strides).  No
    output may overlap an input or another output.
    """
    try:
        dev, dtype = _current_device(), x.dtype
        tokens, width = x.shape
        row, along = x.stride()
        good = dtype in ROW_CODES and along == 1 and x.get_device() == dev
        if gate is not None:
            gate_row, along = gate.stride()
            good = good and gate.dtype is dtype and gate.shape == x.shape and along == 1 and gate.get_device() == dev
    except (AttributeError, TypeError, ValueError, RuntimeError):
        good = False
    if not good:
        _need_rows(x, "x", ROW_CODES, (None, None))
        row = x.stride(0)
        tokens, width = x.shape
        if gate is not None:
            _need_rows(gate, "gate", (x.dtype,), x.shape)
            gate_row = gate.stride(0)
    code, gate_ptr = 0, 0
    if gate is None:
        gate_row = 0
    else:
        code, gate_ptr = ACTIVATIONS.get(activation, 0), gate.data_ptr()
        if not code:
            raise ValueError(f"activation must be {' or '.join(map(repr, ACTIVATIONS))}, got {activation!r}")
    q, scales, q_row, s_row, s_block = _outputs(q, scales, tokens, width, x.device, stream)
    call = _QUANT.pack(x.data_ptr(), gate_ptr, q.data_ptr(), scales.data_ptr(), tokens, width, row, gate_row, q_row,
                       s_row, s_block, ROW_CODES[dtype], code)
    check(_fn("quant_fp8")(call, _current_stream(dev) if stream is None else _streams.handle(stream)))
    return q, scales


def rms_norm_fp8(x, weight, residual=None, *, eps: float = 1e-6, out=None, q=None, scales=None, stream=None):
    """Root-mean-square norm of x + residual, in fp8 with scales: gemm_fp8's operand before a
    layer's projections.

    x, residual: float16 or bfloat16 [tokens, width], rows contiguous, width a multiple of 8 up
    to 32768; weight: [width] of x's type or float32.  With a residual, residual <- x + residual
    (rounded to its type, in place), and the norm is of that; without one it is of x.  out, if
    given, receives the normalised values in x's type too.  Returns (q, scales) as quant_fp8.  No
    output (residual among them) may overlap an input or another output.
    """
    try:
        dev, dtype = _current_device(), x.dtype
        tokens, width = x.shape
        row, along = x.stride()
        good = (dtype in ROW_CODES and along == 1 and x.get_device() == dev and weight.shape == (width,)
                and (weight.dtype is dtype or weight.dtype is _F32) and weight.get_device() == dev and weight.is_contiguous())
        res_ptr = res_row = out_ptr = out_row = 0
        if residual is not None:
            res_row, along = residual.stride()
            res_ptr = residual.data_ptr()
            good = good and along == 1 and residual.dtype is dtype and residual.shape == x.shape and residual.get_device() == dev
        if out is not None:
            out_row, along = out.stride()
            out_ptr = out.data_ptr()
            good = good and along == 1 and out.dtype is dtype and out.shape == x.shape and out.get_device() == dev
    except (AttributeError, TypeError, ValueError, RuntimeError):
        good = False
    if not good:
        _need_rows(x, "x", ROW_CODES, (None, None))
        (tokens, width), row = x.shape, x.stride(0)
        _need(weight, "weight", (x.dtype, _F32), (x.shape[1],))
        if not weight.is_contiguous():
            raise ValueError("weight must be contiguous")
        for name, t in (("residual", residual), ("out", out)):
            if t is not None:
                _need_rows(t, name, (x.dtype,), x.shape)
        # nothing is wrong: a row of one value, say, whose stride may be anything
        res_ptr, res_row = (0, 0) if residual is None else (residual.data_ptr(), residual.stride(0))
        out_ptr, out_row = (0, 0) if out is None else (out.data_ptr(), out.stride(0))
    q, scales, q_row, s_row, s_block = _outputs(q, scales, tokens, width, x.device, stream)
    if not hasattr(eps, "__float__"):
        raise TypeError(f"eps must be a number, got {type(eps).__name__}")
    try:
        call = _NORM.pack(x.data_ptr(), weight.data_ptr(), res_ptr, out_ptr, q.data_ptr(), scales.data_ptr(), tokens, width, row,
                          res_row, out_row, q_row, s_row, s_block, eps, ROW_CODES[dtype], 3 if weight.dtype is _F32 else ROW_CODES[dtype])
    except OverflowError as e:
        raise ValueError(f"eps is out of range: {eps}") from e
    check(_fn("rms_norm_fp8")(call, _current_stream(dev) if stream is None else _streams.handle(stream)))
    return q, scales
