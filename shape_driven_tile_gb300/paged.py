"""The paged key-value cache of a decode step: block tables and slot maps, appending to the
cache, and attention of one new token per request over it.

As in the package's other calls, the functions check and marshal arguments and call the C
entry points of the same names (include/sdt.h); every step runs in the library's kernels on
the current stream, without a synchronisation, so a step can be captured in a CUDA graph.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import SdtError, check, lib, sdt_paged_cache

GROUP = 32  # values per fp16 scale of a q8 cache
DTYPE_CODES = {torch.float16: 0, torch.bfloat16: 1, torch.int8: 2}


# A decode step calls these once a layer, so a call's own time counts: the library's functions
# are looked up once, the current stream is asked for as the raw handle, and a tensor that is
# as it should be passes one comparison.
_current_stream = torch._C._cuda_getCurrentRawStream
_functions = {}


def _fn(name):
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(lib(), name)
    return f


def _stream(stream, device):
    if stream is None:
        return _current_stream(device)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _tensor(t, name, dtype, ndim, device=None):
    """A CUDA tensor on the current device (or on `device`, already known to be it)."""
    if type(t) is torch.Tensor and t.dtype is dtype and t.dim() == ndim and t.get_device() == device:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is None:
        if t.get_device() != torch.cuda.current_device():
            raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")
    elif t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{device}")


def _vector(t, name, dtype, n, device):
    if (type(t) is torch.Tensor and t.dtype is dtype and t.get_device() == device and t.dim() == 1 and t.is_contiguous()
            and (n is None or len(t) == n)):
        return
    _tensor(t, name, dtype, 1, device)
    if n is not None and t.shape[0] != n:
        raise ValueError(f"{name} must have {n} entries, got {t.shape[0]}")
    if t.stride(0) != 1 and t.shape[0] > 1:
        raise ValueError(f"{name} must be contiguous")


class PagedCache:
    """A paged key-value cache: views of the caller's tensors, checked once.

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
            _tensor(t, name, dtype, 4)
            want = tuple(k.shape) if t.dtype is k.dtype else (*k.shape[:3], k.shape[3] // GROUP)
            if tuple(t.shape) != want:
                raise ValueError(f"{name} must be {want}, got {tuple(t.shape)}")
            if t.stride(3) != 1 and t.shape[3] > 1:
                raise ValueError(f"{name} must be contiguous in its last dimension")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.num_pages, self.page_size, self.kv_heads, self.head_dim = k.shape
        self.dtype, self.device_index = k.dtype, k.get_device()
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
        self._ref = ctypes.byref(d)


def _cache(cache):
    if not isinstance(cache, PagedCache):
        raise TypeError("cache must be a PagedCache")
    if cache.device_index != torch._C._cuda_getDevice():
        raise ValueError(f"the cache is on cuda:{cache.device_index}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return cache.device_index


def paged_tables(lens, new_tokens, free_pages, table, *, page_size: int, slots, kv_lens=None, starts=None, used=None,
                 stream=None):
    """Block tables and slot maps of a step, built on the GPU from the requests' lengths.

    lens, new_tokens: int32 [batch], the tokens each request holds and adds.  free_pages: int32,
    the page ids that may be taken, in order.  table: int32 [batch, max_pages], row b naming
    request b's pages; the new tokens' pages are written into it.  slots: int64, filled with
    ``page * page_size + offset`` of the new tokens, request after request, then -1.
    Returns (kv_lens, starts, slots, used): int32 lens + new_tokens, int32 [batch + 1] prefix
    sums of new_tokens, and int32 [1], the pages taken; where that exceeds free_pages' length,
    the entries and slots without a page are -1.
    """
    _tensor(lens, "lens", torch.int32, 1)
    dev, batch = lens.get_device(), lens.shape[0]
    _vector(lens, "lens", torch.int32, batch, dev)
    _vector(new_tokens, "new_tokens", torch.int32, batch, dev)
    _vector(free_pages, "free_pages", torch.int32, None, dev)
    _tensor(table, "table", torch.int32, 2, dev)
    _vector(slots, "slots", torch.int64, None, dev)
    if table.shape[0] != batch or (table.stride(1) != 1 and table.shape[1] > 1):
        raise ValueError(f"table must be [{batch}, max_pages] with contiguous rows")
    if kv_lens is None:
        kv_lens = torch.empty(batch, dtype=torch.int32, device=lens.device)
    else:
        _vector(kv_lens, "kv_lens", torch.int32, batch, dev)
    if starts is None:
        starts = torch.empty(batch + 1, dtype=torch.int32, device=lens.device)
    else:
        _vector(starts, "starts", torch.int32, batch + 1, dev)
    if used is None:
        used = torch.empty(1, dtype=torch.int32, device=lens.device)
    else:
        _vector(used, "used", torch.int32, 1, dev)
    if batch == 0:
        raise SdtError(-3, "paged_tables: batch must be at least 1")
    check(_fn("paged_tables")(batch, page_size, table.shape[1], lens.data_ptr(), new_tokens.data_ptr(),
                             free_pages.data_ptr(), free_pages.shape[0], table.data_ptr(),
                             table.stride(0) if batch > 1 else table.shape[1], kv_lens.data_ptr(), starts.data_ptr(),
                             slots.data_ptr(), slots.shape[0], used.data_ptr(), _stream(stream, dev)))
    return kv_lens, starts, slots, used


def paged_append(k, v, slots, cache: PagedCache, *, stream=None) -> PagedCache:
    """Writes k and v [tokens, kv_heads, head_dim] (float16 or bfloat16; a 16-bit cache's own
    type) into the cache at slots (int64 [tokens], page * page_size + offset; negative: left
    out), as q8 if the cache is.  k and v may be slices of wider rows."""
    dev = _cache(cache)
    dtype = cache.dtype if cache.dtype is not torch.int8 else k.dtype if isinstance(k, torch.Tensor) else None
    if dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("k must be a float16 or bfloat16 tensor")
    _tensor(k, "k", dtype, 3, dev)
    _tensor(v, "v", dtype, 3, dev)
    tokens = k.shape[0]
    want = (tokens, cache.kv_heads, cache.head_dim)
    if k.shape != want or v.shape != want:
        raise ValueError(f"k and v must be {want}, got {tuple(k.shape)} and {tuple(v.shape)}")
    if k.stride(2) != 1 or v.stride(2) != 1:
        raise ValueError("k and v must be contiguous in their last dimension")
    _vector(slots, "slots", torch.int64, tokens, dev)
    check(_fn("paged_append")(tokens, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1),
                             DTYPE_CODES[dtype], slots.data_ptr(), cache._ref, _stream(stream, dev)))
    return cache


def paged_attn_workspace(q_heads: int, kv_heads: int, head_dim: int, device=None) -> torch.Tensor:
    """A zeroed, 256-byte aligned workspace for paged_attn_m1 (owned by the caller; any batch and lengths)."""
    nbytes = int(lib().sdt_paged_attn_workspace_bytes(q_heads, kv_heads, head_dim))
    if nbytes == 0:
        raise SdtError(-3, lib().sdt_last_error().decode())
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=device or "cuda")
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + nbytes]
    check(lib().sdt_splitk_workspace_init(ws.data_ptr(), nbytes, _stream(None, ws.get_device())))
    return ws


def paged_attn_m1(q, cache: PagedCache, table, lens, out=None, *, workspace, scale: float | None = None, window: int = 0,
                  lse=None, stream=None):
    """Attention of one new token per request over the paged cache.

    q: [batch, q_heads, head_dim] float16 or bfloat16 (a 16-bit cache's own type), q_heads a
    multiple of the cache's heads: query head i reads key head i // (q_heads // kv_heads).
    table: int32 [batch, max_pages], lens: int32 [batch].  Request b attends to its tokens
    0 .. lens[b] - 1, or with window > 0 to the last `window` of them; without any it gets
    zeros.  scale: None is 1 / sqrt(head_dim).  lse: float32 [batch, q_heads], if given
    receives log(sum(exp(scores))).  workspace: paged_attn_workspace().
    """
    dev = _cache(cache)
    dtype = cache.dtype if cache.dtype is not torch.int8 else q.dtype if isinstance(q, torch.Tensor) else None
    if dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("q must be a float16 or bfloat16 tensor")
    _tensor(q, "q", dtype, 3, dev)
    batch, q_heads, head_dim = q.shape
    if head_dim != cache.head_dim:
        raise ValueError(f"q has heads of {head_dim}, the cache of {cache.head_dim}")
    qb, qh, qd = q.stride()
    if qd != 1:
        raise ValueError("q must be contiguous in its last dimension")
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else torch.empty(q.shape, dtype=dtype, device=q.device)
        ob, oh = q_heads * head_dim, head_dim
    else:
        _tensor(out, "out", dtype, 3, dev)
        ob, oh, od = out.stride()
        if out.shape != q.shape or od != 1:
            raise ValueError(f"out must be {tuple(q.shape)}, contiguous in its last dimension")
    _tensor(table, "table", torch.int32, 2, dev)
    rows, wide = table.shape
    if rows != batch or (wide > 1 and table.stride(1) != 1):
        raise ValueError(f"table must be [{batch}, max_pages] with contiguous rows")
    _vector(lens, "lens", torch.int32, batch, dev)
    if lse is not None:
        _tensor(lse, "lse", torch.float32, 2, dev)
        if lse.shape != (batch, q_heads) or not lse.is_contiguous():
            raise ValueError(f"lse must be contiguous {(batch, q_heads)}")
    _vector(workspace, "workspace", torch.uint8, None, dev)
    # (a dimension of one never steps: its stride may be anything)
    check(_fn("paged_attn_m1")(batch, q_heads, q.data_ptr(), qb if batch > 1 else 0, qh if q_heads > 1 else 0,
                               DTYPE_CODES[dtype], cache._ref, table.data_ptr(), table.stride(0) if batch > 1 else wide,
                               wide, lens.data_ptr(), window, head_dim ** -0.5 if scale is None else scale,
                               out.data_ptr(), ob if batch > 1 else 0, oh if q_heads > 1 else 0,
                               None if lse is None else lse.data_ptr(), workspace.data_ptr(), len(workspace),
                               _stream(stream, dev)))
    return out
