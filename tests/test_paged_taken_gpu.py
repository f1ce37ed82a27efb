"""paged_tables with the place in the free list on the device: lengths in place, several CTAs, an empty
pool, and a whole decode step that is captured once and replayed by itself."""
import numpy as np
import pytest
import torch

import shape_driven_tile_gb300 as sdt
from _paged_history import History

pytestmark = pytest.mark.gpu


class Plain:
    """The same requests on the host, page by page."""

    def __init__(self, lens, free, table, page):
        self.lens, self.free, self.table, self.page, self.taken = list(lens), list(free), table.copy(), page, 0

    def step(self, new, num_slots):
        slots, needed, wide = [], 0, self.table.shape[1]
        left = len(self.free) - self.taken
        for b, add in enumerate(new):
            n = self.lens[b]
            for j in range(-(-n // self.page), min(-(-(n + add) // self.page), wide)):
                self.table[b, j] = self.free[self.taken + needed] if needed < left else -1
                needed += 1
            for pos in range(n, n + add):
                j = pos // self.page
                slots.append(self.table[b, j] * self.page + pos % self.page if j < wide and self.table[b, j] >= 0 else -1)
            self.lens[b] = n + add
        self.taken += min(needed, left)
        return (slots + [-1] * num_slots)[:num_slots], needed


def check(dev, batch, page, steps, in_place, most, pool=None, seed=0, max_new=3):
    """`steps` steps of 0 .. max_new tokens a request; tables, slots, lengths and the place after each, exactly."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, most, batch).tolist()
    wide = -(-(most + steps * max_new) // page)
    need = sum(-(-n // page) for n in lens)
    ids = rng.permutation(need + (batch * wide if pool is None else pool)).astype(np.int32)
    table = np.full((batch, wide), -7, np.int32)
    at = 0
    for b, n in enumerate(lens):
        held = -(-n // page)
        table[b, :held] = ids[at:at + held]
        at += held
    plain = Plain(lens, ids[at:], table, page)
    i32 = dict(dtype=torch.int32, device=dev)
    on, free = torch.from_numpy(table).to(dev), torch.from_numpy(ids[at:].copy()).to(dev)
    length, taken, new = torch.tensor(lens, **i32), torch.zeros(2, **i32), torch.zeros(batch, **i32)
    kv = length if in_place else torch.zeros(batch, **i32)
    num_slots = batch * max_new
    slots = torch.empty(num_slots, dtype=torch.int64, device=dev)
    for _ in range(steps):
        add = rng.integers(0, max_new + 1, batch)
        new.copy_(torch.from_numpy(add.astype(np.int32)))
        got = sdt.paged_tables(length, new, free, on, page_size=page, slots=slots, kv_lens=kv, taken=taken)
        want, needed = plain.step(add.tolist(), num_slots)
        assert slots.tolist() == want and got[3].item() == needed
        assert got[0] is kv and kv.tolist() == plain.lens and taken.tolist() == [plain.taken, 0]
        np.testing.assert_array_equal(on.cpu().numpy(), plain.table)
        length.copy_(kv)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page", [1, 7, 16])
@pytest.mark.parametrize("batch", [1, 5, 257])
def test_steps(cuda_device, batch, page, in_place):
    check(cuda_device, batch, page, 12, in_place, 40, seed=batch + page)


@pytest.mark.parametrize("max_new", [9, 130])
def test_several_ctas_in_place(cuda_device, max_new):
    """More slots than one CTA is launched for: every CTA still reads the old lengths."""
    check(cuda_device, 700, 16, 6, True, 300, max_new=max_new)


def test_most_requests_in_place(cuda_device):
    check(cuda_device, 16384, 16, 2, True, 50, max_new=2)


@pytest.mark.parametrize("pool", [0, 1, 17])
def test_a_pool_that_runs_out(cuda_device, pool):
    check(cuda_device, 30, 4, 8, True, 20, pool=pool)


def test_a_place_outside_the_list_takes_nothing(cuda_device):
    i32 = dict(dtype=torch.int32, device=cuda_device)
    for place, want in ((5, [-1, 3]), (2, [-1, 2]), (-4, [7, 1])):
        taken, table = torch.tensor([place, 0], **i32), torch.tensor([[-7]], **i32)
        out = sdt.paged_tables(torch.tensor([0], **i32), torch.tensor([1], **i32), torch.tensor([7, 8], **i32), table, page_size=4,
                               slots=torch.empty(1, dtype=torch.int64, device=cuda_device), taken=taken)
        assert table.item() == want[0] and out[2].item() == (want[0] * 4 if want[0] >= 0 else -1)
        assert taken.tolist() == [min(max(place, 0), 2) + (want[0] >= 0), 0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_captured_step_replayed_by_itself(cuda_device, dtype):
    """Tables, append and attention in one graph: between replays only the new rows change."""
    dev, page, heads, qheads, d = cuda_device, 16, 2, 8, 64
    lens, steps = [16, 0, 31, 200, 7], 40
    g = torch.Generator(device=dev).manual_seed(1)
    i32 = dict(dtype=torch.int32, device=dev)
    batch, wide = len(lens), -(-(max(lens) + steps + 1) // page)
    pool = torch.randperm(batch * wide, generator=g, device=dev).to(torch.int32)
    cache = sdt.PagedCache(*(torch.full((len(pool), page, heads, d), float("nan"), dtype=dtype, device=dev) for _ in range(2)))
    table, length, taken = torch.full((batch, wide), -1, **i32), torch.zeros(batch, **i32), torch.zeros(2, **i32)
    rand = lambda n, h: torch.randn(n, h, d, generator=g, device=dev).to(dtype)
    history = History(batch)
    k, v = rand(sum(lens), heads), rand(sum(lens), heads)
    slots = torch.empty(sum(lens), dtype=torch.int64, device=dev)
    sdt.paged_tables(length, torch.tensor(lens, **i32), pool, table, page_size=page, slots=slots, kv_lens=length, taken=taken)
    sdt.paged_append(k, v, slots, cache)
    history.add(k, v, lens)
    k, v, q, out = rand(batch, heads), rand(batch, heads), rand(batch, qheads), torch.zeros(batch, qheads, d, dtype=dtype, device=dev)
    new, slots, lens_out = torch.ones(batch, **i32), torch.empty(batch, dtype=torch.int64, device=dev), list(lens)
    starts, used = torch.empty(batch + 1, **i32), torch.empty(1, **i32)
    ws = sdt.paged_attn_workspace(qheads, heads, d)

    def step():
        sdt.paged_tables(length, new, pool, table, page_size=page, slots=slots, kv_lens=length, starts=starts, used=used, taken=taken)
        sdt.paged_append(k, v, slots, cache)
        sdt.paged_attn_m1(q, cache, table, length, out, workspace=ws)

    step()  # one step as it is, then the captured one
    graph = None
    for i in range(steps):
        if i:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            for t in (k, v, q):
                t.copy_(rand(*t.shape[:2]))
            graph.replay()
        history.add(k, v, [1] * batch)
        lens_out = [n + 1 for n in lens_out]
        want, tol = history.attention(q)
        off = (out.cpu().double() - want).abs()
        assert (off <= tol).all(), f"step {i}: error / bound {(off / tol).max():.3g}"
        assert length.tolist() == lens_out and taken.tolist() == [sum(-(-n // page) for n in lens_out), 0]
    sdt.check_device_status()
    named = table[table >= 0]
    assert named.unique().numel() == named.numel() == taken[0].item()


def test_refusals(cuda_device):
    i32 = dict(dtype=torch.int32, device=cuda_device)
    z = lambda *s: torch.zeros(*s, **i32)
    args = lambda: (z(2), z(2), z(4), z(2, 3))
    kw = dict(page_size=16, slots=torch.zeros(2, dtype=torch.int64, device=cuda_device))
    for taken in (z(1), z(3), z(2, 1), z(4)[::2], z(2).long(), z(2).cpu(), [0, 0]):
        with pytest.raises((TypeError, ValueError)):
            sdt.paged_tables(*args(), **kw, taken=taken)
    lens, new, free, table = args()
    with pytest.raises(sdt.SdtError, match="overlap"):
        sdt.paged_tables(lens, new, free, table, **kw, taken=lens)
    with pytest.raises(sdt.SdtError, match="overlap"):
        sdt.paged_tables(lens, new, free, table, **kw, taken=z(2), kv_lens=new)
    with pytest.raises(sdt.SdtError, match="overlap"):
        sdt.paged_tables(lens, new, free, table, **kw, kv_lens=lens)
