"""What the paged operators refuse on the host, before anything is enqueued (no GPU needed)."""
import ctypes

import pytest
import torch

import shape_driven_tile_gb300 as sdt
from shape_driven_tile_gb300 import _lib, paged

A = 0x10000  # an address that is aligned to everything; never followed
NULL, ALIGN, SHAPE, ARG = -1, -2, -3, -10


def cache(**kw):
    d = _lib.sdt_paged_cache()
    base = dict(k=A, v=A, num_pages=8, page_size=16, kv_heads=2, head_dim=64, dtype=1, k_page=2048, k_token=128, k_head=64,
                v_page=2048, v_token=128, v_head=64)
    if kw.get("dtype") == 2:
        base.update(k_scales=A, v_scales=A, ks_page=64, ks_token=4, ks_head=2, vs_page=64, vs_token=4, vs_head=2)
    for k, v in {**base, **kw}.items():
        setattr(d, k, v)
    return d


def attn(c, **kw):
    a = dict(q=A, out=A, lse=0, table=A, lens=A, cache=ctypes.addressof(c), workspace=A, batch=4, q_heads=8, q_batch=512,
             q_head=64, out_batch=512, out_head=64, table_stride=10, max_pages=10, window=0, workspace_bytes=1 << 30,
             scale=1.0, dtype=1)
    assert not set(kw) - set(a)
    return sdt.lib().paged_attn_m1(paged._ATTN.pack(*(0 if v is None else v for v in {**a, **kw}.values())), None)


def append(c, **kw):
    a = dict(tokens=4, k=A, k_token=128, k_head=64, v=A, v_token=128, v_head=64, dtype=1, slots=A, cache=ctypes.byref(c),
             stream=None)
    assert not set(kw) - set(a)
    return sdt.lib().paged_append(*{**a, **kw}.values())


def tables(**kw):
    a = dict(lens=A, new_tokens=A, free_pages=A, table=A, kv_lens=A, starts=A, used=A, slots=A, batch=4, page_size=16,
             max_pages=10, table_stride=10, num_free=5, num_slots=4)
    assert not set(kw) - set(a)
    return sdt.lib().paged_tables(paged._STEP.pack(*(0 if v is None else v for v in {**a, **kw}.values())), None)


BAD_CACHES = [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=A + 8), ALIGN), (dict(v=A + 2), ALIGN), (dict(dtype=7), ARG),
    (dict(head_dim=0), SHAPE), (dict(head_dim=60), SHAPE), (dict(head_dim=264), SHAPE), (dict(num_pages=0), SHAPE),
    (dict(page_size=0), SHAPE), (dict(kv_heads=0), SHAPE), (dict(kv_heads=65536), SHAPE),
    (dict(num_pages=1 << 27, page_size=16), SHAPE), (dict(page_size=1 << 40), SHAPE), (dict(k_token=-128), ARG),
    (dict(k_head=4), ARG), (dict(v_page=1), ARG),
    (dict(dtype=2, head_dim=32), SHAPE), (dict(dtype=2, head_dim=96), SHAPE), (dict(dtype=2, k_scales=None), NULL),
    (dict(dtype=2, v_scales=A + 2), ALIGN), (dict(dtype=2, ks_head=1), ARG), (dict(dtype=2, k_token=72), ARG),
]


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_caches(change, status):
    assert attn(cache(**change)) == status
    assert append(cache(**change)) == status
    assert sdt.lib().sdt_last_error()


def test_no_cache():
    assert sdt.lib().paged_append(4, A, 128, 64, A, 128, 64, 1, A, None, None) == NULL
    assert attn(cache(), cache=None) == NULL


def test_no_arguments():
    assert sdt.lib().paged_attn_m1(None, None) == NULL and sdt.lib().paged_tables(None, None) == NULL


@pytest.mark.parametrize("change,status", [
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(lens=None), NULL), (dict(table=None), NULL), (dict(workspace=None), NULL),
    (dict(q=A + 2), ALIGN), (dict(out=A + 4), ALIGN), (dict(lens=A + 1), ALIGN), (dict(table=A + 2), ALIGN), (dict(lse=A + 2), ALIGN),
    (dict(workspace=A + 16), ALIGN), (dict(q_head=63), ARG), (dict(q_batch=511), ARG), (dict(out_head=66), ARG),
    (dict(out_batch=513), ARG), (dict(dtype=0), ARG), (dict(dtype=2), ARG), (dict(window=-1), ARG), (dict(batch=-1), SHAPE),
    (dict(batch=(1 << 20) + 1), SHAPE), (dict(q_heads=7), SHAPE), (dict(q_heads=0), SHAPE), (dict(q_heads=1), SHAPE),
    (dict(q_heads=65538), SHAPE), (dict(max_pages=-1), SHAPE), (dict(max_pages=1 << 27), SHAPE), (dict(table_stride=9), ARG),
])
def test_attention(change, status):
    assert attn(cache(), **change) == status
    assert sdt.lib().sdt_last_error()


def test_attention_of_no_request_is_nothing():
    assert attn(cache(), batch=0, q=None, out=None, lens=None, table=None, workspace=None) == 0


@pytest.mark.parametrize("change,status", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(k=A + 2), ALIGN), (dict(v=A + 8), ALIGN),
    (dict(slots=A + 4), ALIGN), (dict(dtype=0), ARG), (dict(dtype=2), ARG), (dict(k_token=4), ARG), (dict(v_head=-8), ARG),
    (dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE),
])
def test_append(change, status):
    assert append(cache(), **change) == status
    assert append(cache(), tokens=0, k=None, v=None, slots=None) == 0


@pytest.mark.parametrize("change,status", [
    (dict(batch=0), SHAPE), (dict(batch=16385), SHAPE), (dict(page_size=0), SHAPE), (dict(max_pages=-1), SHAPE),
    (dict(page_size=1 << 30), SHAPE), (dict(num_free=-1), SHAPE), (dict(num_slots=-1), SHAPE), (dict(num_slots=1 << 31), SHAPE),
    (dict(table_stride=9), ARG), (dict(lens=None), NULL), (dict(new_tokens=None), NULL), (dict(free_pages=None), NULL),
    (dict(table=None), NULL), (dict(kv_lens=None), NULL), (dict(starts=None), NULL), (dict(slots=None), NULL), (dict(used=None), NULL),
    (dict(lens=A + 2), ALIGN), (dict(slots=A + 4), ALIGN), (dict(table=A + 1), ALIGN),
])
def test_tables(change, status):
    assert tables(**change) == status


def test_workspace_of_bad_sizes():
    for sizes in ((7, 2, 64), (2, 4, 64), (8, 0, 64), (8, 2, 264), (8, 2, 0)):
        assert sdt.lib().sdt_paged_attn_workspace_bytes(*sizes) == 0
        assert sdt.lib().sdt_last_error()


def host(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_python_refuses_what_is_not_a_cache_of_tensors():
    for bad in ([1.0], None, host(1, 16, 2, 64, dtype=torch.float32)):
        with pytest.raises(TypeError):
            sdt.PagedCache(bad, bad)
    with pytest.raises(ValueError):  # not on a GPU
        sdt.PagedCache(host(1, 16, 2, 64), host(1, 16, 2, 64))
    with pytest.raises(ValueError):
        sdt.PagedCache(host(1, 16, 2, 64), host(1, 16, 2, 64), host(1, 16, 2, 2), None)
    with pytest.raises(ValueError):
        sdt.PagedCache(host(1, 16, 2, 64, dtype=torch.int8), host(1, 16, 2, 64, dtype=torch.int8))
    for call in (lambda: sdt.paged_append(host(1, 2, 64), host(1, 2, 64), host(1), None),
                 lambda: sdt.paged_attn_m1(host(1, 2, 64), None, host(1, 1), host(1), workspace=None)):
        with pytest.raises(TypeError):
            call()
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError):
        sdt.paged_tables(host(2, **i32), host(2, **i32), host(2, **i32), host(2, 3, **i32), page_size=16,
                         slots=host(2, dtype=torch.int64))
