"""The paged key-value cache of a decode step: block tables and slot maps, appending to the
cache, and attention of one new token per request over it.

As in the package's other calls, the functions check and marshal arguments and call the C
entry points of the same names (include/sdt.h); every step runs in the library's kernels on
the current stream, without a synchronisation, so a step can be captured in a CUDA graph.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import _streams
from ._lib import SdtError, check, lib, sdt_paged_cache

GROUP = 32  # values per fp16 scale of a q8 cache
DTYPE_CODES = {torch.float16: 0, torch.bfloat16: 1, torch.int8: 2}


# A decode step calls these once a layer, so a call's own time counts.  The library's functions
# are looked up once, the current stream is asked for as the raw handle, and each call first
# compares everything in one expression; only if something is not plainly as it should be, the
# _need_* functions go through it again and raise what is wrong.
_current_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_I32, _I64 = torch.int32, torch.int64
# sdt_paged_step and sdt_paged_attn (include/sdt.h): packing them takes a fraction of what ctypes takes
# for as many arguments
_STEP, _ATTN = struct.Struct("8P6q"), struct.Struct("7P10qfi")
_FLT_MAX = 3.4028234663852886e38
_functions = {}


def _fn(name):
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(lib(), name)
    return f


def _refuse(error, **integers):
    """Raises what is wrong with the caller's own numbers, which could not be packed."""
    scale = integers.pop("scale", None)
    for name, value in integers.items():
        if not hasattr(value, "__index__"):
            raise TypeError(f"{name} must be an integer, got {type(value).__name__}") from error
        if not -2 ** 63 <= value < 2 ** 63:
            raise ValueError(f"{name} is out of range: {value}") from error
    if scale is not None and not hasattr(scale, "__float__"):
        raise TypeError(f"scale must be a number, got {type(scale).__name__}") from error
    raise error


def _need(t, name, dtype, ndim):
    """A CUDA tensor on the current device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != _current_device():
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{_current_device()}")


def _need_vector(t, name, dtype, n=None):
    _need(t, name, dtype, 1)
    if n is not None and t.shape[0] != n:
        raise ValueError(f"{name} must have {n} entries, got {t.shape[0]}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_table(table, batch):
    _need(table, "table", _I32, 2)
    if table.shape[0] != batch or (table.stride(1) != 1 and table.shape[1] > 1):
        raise ValueError(f"table must be [{batch}, max_pages] with contiguous rows")


def _need_cache(cache):
    if not isinstance(cache, PagedCache):
        raise TypeError("cache must be a PagedCache")
    if cache.device_index != _current_device():
        raise ValueError(f"the cache is on cuda:{cache.device_index}, but the current device is cuda:{_current_device()}")


def _need_values(t, name, cache, shape):
    """Queries, keys or values [n, heads, head_dim] of a type that goes with the cache."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in cache.value_dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, cache.value_dtypes))}, got {t.dtype}")
    _need(t, name, t.dtype, 3)
    for have, want in zip(t.shape, shape):
        if want is not None and have != want:
            raise ValueError(f"{name} must be {tuple('any' if w is None else w for w in shape)}, got {tuple(t.shape)}")
    if t.stride(2) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


class PagedCache:
    """A paged key-value cache: views of the caller's tensors, whose types and shapes are checked once (widths,
    alignment and strides with each call).

    k, v: [num_pages, page_size, kv_heads, head_dim], float16, bfloat16 or int8, any strides
    with head_dim contiguous (a cache that is laid out head by head is given as
    ``t.transpose(1, 2)``).  int8 keys and values (q8) come with k_scales and v_scales, float16
    [num_pages, page_size, kv_heads, head_dim // 32]: element e of a head is
    ``q[e] * scale[e // 32]``.  head_dim is a multiple of 8 (q8: of 64) up to 256.
    """

    def __init__(self, k, v, k_scales=None, v_scales=None):
        if not isinstance(k, torch.Tensor) or k.dtype not in DTYPE_CODES:
            raise TypeError("k must be a float16, bfloat16 or int8 tensor")
        q8 = k.dtype is torch.int8
        tensors = [("k", k, k.dtype), ("v", v, k.dtype)]
        if (k_scales is not None) != q8 or (v_scales is not None) != q8:
            raise ValueError("k_scales and v_scales go with an int8 cache, and only with one")
        if q8:
            tensors += [("k_scales", k_scales, torch.float16), ("v_scales", v_scales, torch.float16)]
        for name, t, dtype in tensors:
            _need(t, name, dtype, 4)
            want = tuple(k.shape) if t.dtype is k.dtype else (*k.shape[:3], k.shape[3] // GROUP)
            if tuple(t.shape) != want:
                raise ValueError(f"{name} must be {want}, got {tuple(t.shape)}")
            if t.stride(3) != 1 and t.shape[3] > 1:
                raise ValueError(f"{name} must be contiguous in its last dimension")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.num_pages, self.page_size, self.kv_heads, self.head_dim = k.shape
        self.dtype, self.device_index = k.dtype, k.get_device()
        self.value_dtypes = (torch.float16, torch.bfloat16) if q8 else (k.dtype,)  # of queries and new values
        d = sdt_paged_cache()
        d.num_pages, d.page_size, d.kv_heads, d.head_dim = k.shape
        d.dtype = DTYPE_CODES[k.dtype]
        for name, short, t in (("k", "k", k), ("v", "v", v), ("k_scales", "ks", k_scales), ("v_scales", "vs", v_scales)):
            if t is not None:
                setattr(d, name, t.data_ptr())
                for axis, dim in (("page", 0), ("token", 1), ("head", 2)):
                    # a dimension of one never steps
                    setattr(d, f"{short}_{axis}", t.stride(dim) if t.shape[dim] > 1 else 0)
        self.descriptor = d
        self._ref, self._address = ctypes.byref(d), ctypes.addressof(d)


def paged_tables(lens, new_tokens, free_pages, table, *, page_size: int, slots, kv_lens=None, starts=None, used=None,
                 taken=None, stream=None):
    """Block tables and slot maps of a step, built on the GPU from the requests' lengths.

    lens, new_tokens: int32 [batch], the tokens each request holds and adds.  free_pages: int32,
    the page ids that may be taken, in order.  table: int32 [batch, max_pages], row b naming
    request b's pages; the new tokens' pages are written into it.  slots: int64, filled with
    ``page * page_size + offset`` of the new tokens, request after request, then -1.
    Returns (kv_lens, starts, slots, used): int32 lens + new_tokens, int32 [batch + 1] prefix
    sums of new_tokens, and int32 [1], the pages taken; where that exceeds free_pages' length,
    the entries and slots without a page are -1.  No output may overlap an input or another output.
    taken: int32 [2], zeros at first, for a step that is captured and replayed: taken[0] entries of
    free_pages have been used by earlier calls, the call takes its pages from there on and moves it;
    taken[1] belongs to the kernel.  With it kv_lens may be lens, which is then updated in place.
    """
    try:
        batch, dev = len(lens), _current_device()
        rows, wide = table.shape
        step, along = table.stride()
        good = (rows == batch and (along == 1 or wide <= 1)
                and lens.dtype is _I32 and new_tokens.dtype is _I32 and free_pages.dtype is _I32
                and table.dtype is _I32 and slots.dtype is _I64
                and lens.get_device() == dev and new_tokens.get_device() == dev and free_pages.get_device() == dev
                and table.get_device() == dev and slots.get_device() == dev
                and lens.dim() == 1 and new_tokens.shape == lens.shape and free_pages.dim() == 1 and slots.dim() == 1
                and lens.is_contiguous() and new_tokens.is_contiguous() and free_pages.is_contiguous()
                and slots.is_contiguous())
    except (AttributeError, TypeError, ValueError, RuntimeError):
        good = False
    if not good:
        _need_vector(lens, "lens", _I32)
        batch = len(lens)
        _need_vector(new_tokens, "new_tokens", _I32, batch)
        _need_vector(free_pages, "free_pages", _I32)
        _need_table(table, batch)
        _need_vector(slots, "slots", _I64)
    if kv_lens is None:
        kv_lens = torch.empty_like(lens) if stream is None else _streams.empty(batch, _I32, lens.device, stream)
    else:
        _need_vector(kv_lens, "kv_lens", _I32, batch)
    if starts is None:
        starts = _streams.empty(batch + 1, _I32, lens.device, stream)
    else:
        _need_vector(starts, "starts", _I32, batch + 1)
    if used is None:
        used = _streams.empty(1, _I32, lens.device, stream)
    else:
        _need_vector(used, "used", _I32, 1)
    try:
        call = _STEP.pack(lens.data_ptr(), new_tokens.data_ptr(), free_pages.data_ptr(), table.data_ptr(), kv_lens.data_ptr(),
                          starts.data_ptr(), used.data_ptr(), slots.data_ptr(), batch, page_size, wide,
                          step if batch > 1 else wide, len(free_pages), len(slots))
    except (struct.error, TypeError, ValueError, OverflowError) as e:
        _refuse(e, page_size=page_size)
    on = _current_stream(dev) if stream is None else _streams.handle(stream)
    if taken is None:
        check(_fn("paged_tables")(call, on))
    else:
        _need_vector(taken, "taken", _I32, 2)
        check(_fn("paged_tables_taken")(call, taken.data_ptr(), on))
    return kv_lens, starts, slots, used


def paged_append(k, v, slots, cache: PagedCache, *, stream=None) -> PagedCache:
    """Writes k and v [tokens, kv_heads, head_dim] (float16 or bfloat16; a 16-bit cache's own
    type) into the cache at slots (int64 [tokens], page * page_size + offset; negative: left
    out), as q8 if the cache is.  k and v may be slices of wider rows.  Slots that are not
    negative must differ: tokens with one slot may leave a row mixed from both."""
    try:
        dev, dtype, tokens = cache.device_index, k.dtype, len(k)
        want = (tokens, cache.kv_heads, cache.head_dim)
        kt, kh, kd = k.stride()
        vt, vh, vd = v.stride()
        good = (dev == _current_device() and dtype in cache.value_dtypes and v.dtype is dtype and slots.dtype is _I64
                and k.get_device() == dev and v.get_device() == dev and slots.get_device() == dev
                and k.shape == want and v.shape == want and slots.shape == want[:1] and kd == 1 and vd == 1
                and slots.is_contiguous())
    except (AttributeError, TypeError, ValueError, RuntimeError):
        good = False
    if not good:
        _need_cache(cache)
        _need_values(k, "k", cache, (None, cache.kv_heads, cache.head_dim))
        _need_values(v, "v", cache, k.shape)
        if v.dtype is not k.dtype:
            raise TypeError("k and v must have one type")
        _need_vector(slots, "slots", _I64, len(k))
    check(_fn("paged_append")(tokens, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, DTYPE_CODES[dtype], slots.data_ptr(),
                              cache._ref, _current_stream(dev) if stream is None else _streams.handle(stream)))
    return cache


def paged_attn_workspace(q_heads: int, kv_heads: int, head_dim: int, device=None) -> torch.Tensor:
    """A 256-byte aligned workspace for paged_attn_m1 (owned by the caller; any batch and lengths).  Its counters
    are zeroed on the current stream, which a first call on another stream has to wait for."""
    nbytes = int(lib().sdt_paged_attn_workspace_bytes(q_heads, kv_heads, head_dim))
    if nbytes == 0:
        raise SdtError(-3, lib().sdt_last_error().decode())
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=device or "cuda")
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + nbytes]
    check(lib().sdt_splitk_workspace_init(ws.data_ptr(), nbytes, _current_stream(ws.get_device())))
    return ws


def paged_attn_m1(q, cache: PagedCache, table, lens, out=None, *, workspace, scale: float | None = None, window: int = 0,
                  lse=None, stream=None):
    """Attention of one new token per request over the paged cache.

    q: [batch, q_heads, head_dim] float16 or bfloat16 (a 16-bit cache's own type), q_heads a
    multiple of the cache's heads: query head i reads key head i // (q_heads // kv_heads).
    table: int32 [batch, max_pages], lens: int32 [batch].  Request b attends to its tokens
    0 .. lens[b] - 1, or with window > 0 to the last `window` of them; without any it gets
    zeros.  A request that names a page outside the cache gets NaN (and check_device_status()
    reports it).  scale: None is 1 / sqrt(head_dim).  lse: float32 [batch, q_heads], if given
    receives log(sum(exp(scores))).  workspace: paged_attn_workspace().
    """
    try:
        dev, dtype = cache.device_index, q.dtype
        batch, q_heads, head_dim = q.shape
        rows, wide = table.shape
        qb, qh, qd = q.stride()
        step, along = table.stride()
        good = (dev == _current_device() and dtype in cache.value_dtypes and head_dim == cache.head_dim and qd == 1
                and rows == batch and (along == 1 or wide <= 1)
                and table.dtype is _I32 and lens.dtype is _I32 and workspace.dtype is torch.uint8
                and q.get_device() == dev and table.get_device() == dev and lens.get_device() == dev
                and workspace.get_device() == dev and lens.dim() == 1 and len(lens) == batch and workspace.dim() == 1
                and lens.is_contiguous() and workspace.is_contiguous())
    except (AttributeError, TypeError, ValueError, RuntimeError):
        good = False
    if not good:
        _need_cache(cache)
        _need_values(q, "q", cache, (None, None, cache.head_dim))
        _need_table(table, len(q))
        _need_vector(lens, "lens", _I32, len(q))
        _need_vector(workspace, "workspace", torch.uint8)
    if out is None:
        out = torch.empty_like(q) if stream is None and q.is_contiguous() else _streams.empty(q.shape, dtype, q.device, stream)
        ob, oh = q_heads * head_dim, head_dim
    else:
        _need(out, "out", dtype, 3)
        ob, oh, od = out.stride()
        if out.shape != q.shape or od != 1:
            raise ValueError(f"out must be {tuple(q.shape)}, contiguous in its last dimension")
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
        if lse.shape != (batch, q_heads) or not lse.is_contiguous():
            raise ValueError(f"lse must be contiguous {(batch, q_heads)}")
    try:  # (a dimension of one never steps: its stride may be anything)
        if scale is None:
            scale = head_dim ** -0.5
        elif _FLT_MAX < abs(scale) < math.inf:
            raise ValueError(f"scale is out of range: {scale}")
        call = _ATTN.pack(
            q.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(), table.data_ptr(), lens.data_ptr(), cache._address,
            workspace.data_ptr(), batch, q_heads, qb if batch > 1 else 0, qh if q_heads > 1 else 0, ob if batch > 1 else 0,
            oh if q_heads > 1 else 0, step if batch > 1 else wide, wide, window, len(workspace), scale, DTYPE_CODES[dtype])
    except (struct.error, TypeError, ValueError, OverflowError) as e:
        _refuse(e, window=window, scale=scale)
    check(_fn("paged_attn_m1")(call, _current_stream(dev) if stream is None else _streams.handle(stream)))
    return out
