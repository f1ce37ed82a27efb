"""paged_tables and paged_append against plain statements of what they write, bit for bit."""
import numpy as np
import pytest
import torch

import shape_driven_tile_gb300 as sdt

pytestmark = pytest.mark.gpu


def tables_ref(lens, new, free, table, page, num_slots):
    table = table.copy()
    wide, taken, slots = table.shape[1], 0, []
    for b, (n, add) in enumerate(zip(lens, new)):
        n, add = min(max(n, 0), wide * page), max(add, 0)
        for j in range(-(-n // page), min(-(-(n + add) // page), wide)):
            table[b, j] = free[taken] if taken < len(free) else -1
            taken += 1
        for pos in range(n, n + add):
            j = pos // page
            slots.append(table[b, j] * page + pos % page if j < wide and table[b, j] >= 0 else -1)
    kv = [min(max(n, 0), wide * page) + max(a, 0) for n, a in zip(lens, new)]
    starts = np.concatenate([[0], np.cumsum(np.maximum(new, 0))])
    slots = (slots + [-1] * num_slots)[:num_slots]
    return kv, starts, slots, taken, table


def check_tables(dev, lens, new, page, wide=None, spare=4, num_slots=None, seed=0):
    rng = np.random.default_rng(seed)
    lens, new = np.asarray(lens, np.int32), np.asarray(new, np.int32)
    need = int(sum(-(-(max(a, 0) + max(b, 0)) // page) for a, b in zip(lens.tolist(), new.tolist())))
    wide = wide or max(1, int(max(-(-(max(a, 0) + max(b, 0)) // page) for a, b in zip(lens.tolist(), new.tolist()))))
    ids = rng.permutation(need + abs(spare) + 1).astype(np.int32)
    table = np.full((len(lens), wide), -7, np.int32)
    at = 0
    for b, n in enumerate(lens.tolist()):
        held = min(-(-max(n, 0) // page), wide)
        table[b, :held] = ids[at:at + held]
        at += held
    free = ids[at:] if spare >= 0 else ids[at:at + max(0, need - at + spare)]
    num_slots = int(np.maximum(new, 0).sum()) + 5 if num_slots is None else num_slots
    kv, starts, slots, taken, want = tables_ref(lens.tolist(), new.tolist(), free.tolist(), table, page, num_slots)
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev)
    td = t(table)
    for _ in range(2):  # the same call writes the same again
        out = sdt.paged_tables(t(lens), t(new), t(free), td, page_size=page,
                               slots=torch.full((num_slots,), 99, dtype=torch.int64, device=dev))
        for got, ref in zip([*out, td], [kv, starts, slots, [taken], want]):
            np.testing.assert_array_equal(got.cpu().numpy(), np.asarray(ref))


@pytest.mark.parametrize("page", [1, 2, 7, 16, 20, 64, 4096])
@pytest.mark.parametrize("batch", [1, 2, 31, 255, 256, 257, 700])
def test_tables(cuda_device, page, batch):
    rng = np.random.default_rng(batch * 100 + page)
    lens = rng.integers(0, 200, batch)
    new = rng.choice([0, 1, 1, 1, 40], batch)
    check_tables(cuda_device, lens, new, page, seed=batch)


def test_tables_of_prompts(cuda_device):
    check_tables(cuda_device, [0, 5, 0, 1000], [9000, 1, 0, 3333], 16)
    check_tables(cuda_device, [0], [20000], 1)


def test_tables_nothing_new(cuda_device):
    check_tables(cuda_device, [3, 0, 16], [0, 0, 0], 16)


def test_tables_short_of_pages_rows_or_slots(cuda_device):
    check_tables(cuda_device, [10, 16, 31], [1, 1, 40], 16, spare=-2)
    check_tables(cuda_device, [10, 16, 31], [1, 1, 40], 16, spare=-100)
    check_tables(cuda_device, [10, 16, 31], [1, 1, 40], 16, wide=2)
    check_tables(cuda_device, [10, 16, 31], [10, 1, 40], 16, num_slots=7)
    check_tables(cuda_device, [10, 16, 31], [10, 1, 40], 16, num_slots=0)


def test_tables_odd_lengths(cuda_device):
    check_tables(cuda_device, [-3, 5, 70], [4, -2, 3], 16, wide=3)


def test_tables_most_requests(cuda_device):
    check_tables(cuda_device, np.arange(16384) % 50, np.arange(16384) % 3, 16)


def test_tables_given_outputs(cuda_device):
    i32 = dict(dtype=torch.int32, device=cuda_device)
    kv, st, us = torch.empty(2, **i32), torch.empty(3, **i32), torch.empty(1, **i32)
    out = sdt.paged_tables(torch.tensor([3, 16], **i32), torch.tensor([1, 1], **i32), torch.tensor([9], **i32),
                           torch.tensor([[4, 0, 0], [5, 0, 0]], **i32), page_size=16,
                           slots=torch.empty(2, dtype=torch.int64, device=cuda_device), kv_lens=kv, starts=st, used=us)
    assert out[0] is kv and out[1] is st and out[3] is us
    assert kv.tolist() == [4, 17] and st.tolist() == [0, 1, 2] and us.tolist() == [1] and out[2].tolist() == [67, 144]


def q8_ref(x):
    """(int8 [..., D], fp16 [..., D / 32]) of fp32 x by the stated rule, in numpy's fp32."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    s = np.minimum(np.abs(np.nan_to_num(g, nan=0.0, posinf=np.inf, neginf=-np.inf)).max(-1) * np.float32(1 / 127),
                   np.float32(65504)).astype(np.float16)
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.rint(g / s.astype(np.float32)[..., None])
    q = np.where((s[..., None] == 0) | np.isnan(g), 0, np.clip(r, -127, 127)).astype(np.int8)
    return q.reshape(x.shape), s


def append_case(dev, tokens, heads, d, page, dtype, q8, layout, seed=0, values=None, pad=0):
    rng = np.random.default_rng(seed)
    pages = -(-tokens // page) + 2
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn(tokens, (2 * heads + 3) * d, generator=g).to(dtype) if values is None else values
    k, v = rows[:, d:(1 + heads) * d].unflatten(1, (heads, d)), rows[:, (2 + heads) * d:(2 + 2 * heads) * d].unflatten(1, (heads, d))
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    if pad:
        slots[::pad] = -1 - np.arange(len(slots[::pad]))
    cdt = torch.int8 if q8 else dtype

    def empty(width, dt):
        shape = (pages, heads, page, width) if layout == "head" else (pages, page, heads, width)
        t = torch.full(shape, 3, dtype=dt, device=dev)
        return t.transpose(1, 2) if layout == "head" else t

    on = [empty(d, cdt), empty(d, cdt)] + ([empty(d // 32, torch.float16), empty(d // 32, torch.float16)] if q8 else [])
    r = rows.to(dev)
    kd, vd = r[:, d:(1 + heads) * d].unflatten(1, (heads, d)), r[:, (2 + heads) * d:(2 + 2 * heads) * d].unflatten(1, (heads, d))
    cache = sdt.PagedCache(*on)
    assert sdt.paged_append(kd, vd, torch.from_numpy(slots).to(dev), cache) is cache
    sdt.check_device_status()
    keep = slots >= 0
    at, off = slots[keep] // page, slots[keep] % page
    for i, x in enumerate((k, v)):
        if q8:
            q, s = q8_ref(x.float().numpy())
            parts = [(on[i], q), (on[2 + i], s)]
        else:
            parts = [(on[i], x)]
        for got, ref in parts:
            want = torch.full(got.shape, 3, dtype=got.dtype)
            want[torch.from_numpy(at), torch.from_numpy(off)] = torch.as_tensor(ref)[torch.from_numpy(keep)].to(got.dtype)
            bits = torch.int8 if got.dtype is torch.int8 else torch.int16
            assert torch.equal(got.cpu().contiguous().view(bits), want.view(bits))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("tokens,heads,d,page", [(1, 1, 8, 1), (1, 8, 128, 16), (7, 5, 40, 3), (65, 32, 128, 16), (3001, 2, 64, 20),
                                                 (513, 3, 256, 64), (129, 1, 248, 7)])
def test_append(cuda_device, tokens, heads, d, page, dtype, layout):
    append_case(cuda_device, tokens, heads, d, page, dtype, False, layout, seed=tokens)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("tokens,heads,d,page", [(1, 1, 64, 1), (1, 8, 128, 16), (65, 3, 192, 16), (3001, 2, 64, 20), (257, 3, 256, 64)])
def test_append_q8(cuda_device, tokens, heads, d, page, dtype, layout):
    append_case(cuda_device, tokens, heads, d, page, dtype, True, layout, seed=tokens)


def test_append_leaves_negative_slots_out(cuda_device):
    append_case(cuda_device, 100, 2, 64, 16, torch.bfloat16, False, "token", pad=3)
    append_case(cuda_device, 100, 2, 64, 16, torch.bfloat16, True, "head", pad=7)
    append_case(cuda_device, 5, 2, 64, 16, torch.bfloat16, True, "head", pad=1)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_append_q8_extreme_values(cuda_device, dtype):
    d = 64
    x = torch.zeros(8, 5 * d)
    x[0] = 1e-9                      # a scale that rounds to zero
    x[1] = 3e-6                      # a subnormal scale: the quotient passes 127
    x[2] = 65504.0
    x[3, ::3] = float("inf")
    x[4, ::5] = float("nan")
    x[4, 1::5] = 2.0
    x[5, ::2] = -float("inf")
    x[6] = torch.arange(5 * d) % 255 - 127.0   # ties and exact quotients
    x[7] = -0.0
    append_case(cuda_device, 8, 1, d, 4, dtype, True, "token", values=x.to(dtype))
    if dtype is torch.bfloat16:
        append_case(cuda_device, 8, 1, d, 4, dtype, True, "token", values=(x * 1e30).to(dtype))


def test_append_slot_past_the_cache_is_reported(cuda_device):
    k = torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16, device=cuda_device)
    v, x = torch.zeros_like(k), torch.ones(3, 1, 64, dtype=torch.bfloat16, device=cuda_device)
    sdt.paged_append(x, x, torch.tensor([5, 32, 2 ** 40], device=cuda_device), sdt.PagedCache(k, v))
    with pytest.raises(sdt.SdtError, match="slot"):
        sdt.check_device_status()
    assert int(k.sum()) == 64 and int(v.sum()) == 64 and (k[0, 5] == 1).all()


def test_append_nothing(cuda_device):
    k = torch.zeros(2, 16, 1, 64, dtype=torch.float16, device=cuda_device)
    x = torch.zeros(0, 1, 64, dtype=torch.float16, device=cuda_device)
    sdt.paged_append(x, x, torch.empty(0, dtype=torch.int64, device=cuda_device), sdt.PagedCache(k, torch.zeros_like(k)))


def test_python_refusals(cuda_device):
    dev, bf = cuda_device, torch.bfloat16
    z = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype, device=dev)
    i32, i64 = torch.int32, torch.int64
    cache = sdt.PagedCache(z(4, 16, 2, 64), z(4, 16, 2, 64))
    with pytest.raises(ValueError):
        sdt.PagedCache(z(4, 16, 2, 64), z(4, 16, 2, 32))
    with pytest.raises(TypeError):
        sdt.PagedCache(z(4, 16, 2, 64), z(4, 16, 2, 64, dtype=torch.float16))
    with pytest.raises(ValueError, match="last dimension"):
        sdt.PagedCache(z(4, 16, 64, 2).transpose(2, 3), z(4, 16, 2, 64))
    bad = sdt.PagedCache(z(4, 16, 2, 60), z(4, 16, 2, 60))  # the library refuses the width
    with pytest.raises(sdt.SdtError, match="head_dim"):
        sdt.paged_append(z(1, 2, 60), z(1, 2, 60), z(1, dtype=i64), bad)
    x, slots = z(3, 2, 64), z(3, dtype=i64)
    for args, err in [((x, z(3, 2, 32), slots), ValueError), ((x, x.half(), slots), TypeError), ((x, x, slots[:2]), ValueError),
                      ((x, x, slots.int()), TypeError), ((x.cpu(), x, slots), ValueError), ((x, x, slots.cpu()), ValueError),
                      ((z(3, 64, 2).transpose(1, 2), x, slots), ValueError), ((x, x, z(6, dtype=i64)[::2]), ValueError),
                      ((x.float(), x, slots), TypeError)]:
        with pytest.raises(err):
            sdt.paged_append(*args, cache)
    q, table, lens, ws = z(3, 4, 64), z(3, 2, dtype=i32), z(3, dtype=i32), sdt.paged_attn_workspace(4, 2, 64)
    for args, kw, err in [
            ((q.half(), cache, table, lens), {}, TypeError), ((z(3, 4, 32), cache, table, lens), {}, ValueError),
            ((z(3, 5, 64), cache, table, lens), {}, sdt.SdtError), ((q, cache, table[:2], lens), {}, ValueError),
            ((q, cache, table.long(), lens), {}, TypeError), ((q, cache, table, lens[:2]), {}, ValueError),
            ((q, cache, table, lens, z(3, 4, 32)), {}, ValueError), ((q, cache, table, lens, q.float()), {}, TypeError),
            ((q, cache, table, lens), dict(lse=z(3, 4)), TypeError),
            ((q, cache, table, lens), dict(lse=z(3, 5, dtype=torch.float32)), ValueError),
            ((q, cache, table, lens), dict(window=-1), sdt.SdtError), ((q, cache, table.t().contiguous().t(), lens), {}, ValueError)]:
        with pytest.raises(err):
            sdt.paged_attn_m1(*args, workspace=ws, **kw)
    for w in (None, ws.cpu(), ws[1:], ws[: 1 << 20], ws.float()):
        with pytest.raises((TypeError, ValueError, sdt.SdtError)):
            sdt.paged_attn_m1(q, cache, table, lens, workspace=w)
    ok = dict(page_size=16, slots=z(3, dtype=i64))
    for args, kw in [((lens, lens[:2], lens, table), {}), ((lens, lens, lens, table[:2]), {}), ((lens, lens, lens.long(), table), {}),
                     ((lens, lens, lens, table), dict(slots=z(3, dtype=i32))), ((lens, lens, lens, table), dict(page_size=0)),
                     ((lens, lens, lens, table), dict(starts=lens)), ((lens[:0], lens[:0], lens, table[:0]), {})]:
        with pytest.raises((TypeError, ValueError, sdt.SdtError)):
            sdt.paged_tables(*args, **{**ok, **kw})
