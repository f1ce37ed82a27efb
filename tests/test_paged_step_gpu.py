"""A whole decode step, tables -> append -> attention, with nothing between the calls: each reads what
the kernel right before it wrote (lengths, table, slots, keys), launched while that one still runs."""
import pytest
import torch

import shape_driven_tile_gb300 as sdt
from _paged_history import History

pytestmark = pytest.mark.gpu
PAGE, HEADS, QHEADS, D = 16, 2, 8, 64


class Step:
    """The buffers of a step, at fixed addresses, and the calls on them."""

    def __init__(self, dev, lens, steps, dtype, seed=0):
        self.g = torch.Generator(device=dev).manual_seed(seed)
        i32 = dict(dtype=torch.int32, device=dev)
        batch = len(lens)
        wide = max(-(-(n + steps) // PAGE) for n in lens)
        self.pages = torch.randperm(batch * wide + 3, generator=self.g, device=dev).to(torch.int32)
        cache = [torch.full((len(self.pages), PAGE, HEADS, D), float("nan"), dtype=dtype, device=dev) for _ in range(2)]
        self.cache, self.workspace = sdt.PagedCache(*cache), sdt.paged_attn_workspace(QHEADS, HEADS, D)
        self.table = torch.full((batch, wide), -1, **i32)
        self.free, self.taken = self.pages.clone(), 0
        self.lens, self.kv_lens = torch.zeros(batch, **i32), torch.zeros(batch, **i32)
        self.starts, self.used = torch.zeros(batch + 1, **i32), torch.zeros(1, **i32)
        self.new = torch.ones(batch, **i32)
        self.slots = torch.zeros(batch, dtype=torch.int64, device=dev)
        self.k, self.v = (torch.zeros(batch, HEADS, D, dtype=dtype, device=dev) for _ in range(2))
        self.q, self.out = (torch.zeros(batch, QHEADS, D, dtype=dtype, device=dev) for _ in range(2))
        self.history, self.dtype, self.dev = History(batch), dtype, dev
        # the prompts
        k, v = self.random(sum(lens), HEADS), self.random(sum(lens), HEADS)
        new = torch.tensor(lens, **i32)
        slots = torch.empty(sum(lens), dtype=torch.int64, device=dev)
        sdt.paged_tables(self.lens, new, self.free, self.table, page_size=PAGE, slots=slots, kv_lens=self.kv_lens)
        sdt.paged_append(k, v, slots, self.cache)
        self.history.add(k, v, lens)
        self.host = list(lens)
        self.taken = sum(-(-n // PAGE) for n in lens)

    def random(self, n, heads):
        return torch.randn(n, heads, D, generator=self.g, device=self.dev).to(self.dtype)

    def feed(self):
        """What changes before a step: the inputs, the lengths, the front of the free list."""
        self.lens.copy_(self.kv_lens)
        self.free[:len(self.pages) - self.taken].copy_(self.pages[self.taken:])
        for t in (self.k, self.v, self.q):
            t.copy_(self.random(*t.shape[:2]))

    def calls(self):
        sdt.paged_tables(self.lens, self.new, self.free, self.table, page_size=PAGE, slots=self.slots, kv_lens=self.kv_lens,
                         starts=self.starts, used=self.used)
        sdt.paged_append(self.k, self.v, self.slots, self.cache)
        sdt.paged_attn_m1(self.q, self.cache, self.table, self.kv_lens, self.out, workspace=self.workspace)

    def after(self):
        self.taken += sum(n % PAGE == 0 for n in self.host)
        self.host = [n + 1 for n in self.host]
        self.history.add(self.k, self.v, [1] * len(self.host))
        want, tol = self.history.attention(self.q)
        off = (self.out.cpu().double() - want).abs()
        assert (off <= tol).all(), f"lengths {self.host}: error / bound {(off / tol).max():.3g}"
        assert self.kv_lens.tolist() == self.host


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("captured", [False, True])
def test_steps_over_page_borders(cuda_device, captured, dtype):
    steps = 20
    step = Step(cuda_device, [16, 0, 31, 200, 7], steps, dtype)
    run = step.calls
    if captured:
        step.feed()
        before = [t.clone() for t in (step.table, step.kv_lens, step.cache.k, step.cache.v)]
        step.calls()  # whatever a first call sets up
        torch.cuda.synchronize()
        for t, x in zip((step.table, step.kv_lens, step.cache.k, step.cache.v), before):
            t.copy_(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step.calls()
        run = graph.replay
    for _ in range(steps):
        step.feed()
        run()
        step.after()
    sdt.check_device_status()
