"""Attention layer of a decode loop on the paged cache: prompts in, then one token a step.

Each step runs, on one stream and without a synchronisation:

  gemm_ex         the fused q, k and v projection of the batch's new rows
  paged_tables    block tables and slots of the new tokens, from the requests' lengths
  paged_append    their keys and values into the cache (16 bits, or q8)
  paged_attn_m1   attention of each request's new token over its cache
  gemm_ex         the output projection

The default layer is the one whose fused projection the repository's decode benchmark
multiplies: width 4096, 32 heads of 128 (K = 4096, N = 12288).  Weights and inputs are
random.  Lengths, pages and the place in the free list are kept on the GPU, so with --graph one
captured step is replayed for all.

    python examples/paged_decode.py [--batch 16] [--prompt 1000] [--steps 32] [--kv-heads 32] [--q8] [--graph]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import shape_driven_tile_gb300 as sdt  # noqa: E402


class Layer:
    """One attention layer's weights, its pages and what it knows of its requests."""

    def __init__(self, batch, max_tokens, *, width=4096, heads=32, kv_heads=32, head_dim=128, page=16, dtype=torch.bfloat16,
                 q8=False, seed=0, device="cuda"):
        self.heads, self.kv_heads, self.head_dim, self.page = heads, kv_heads, head_dim, page
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, k):  # stored [N, K]; its transpose is the product's right operand
            return (torch.randn(n, k, generator=g, device=device) * k ** -0.5).to(dtype)

        self.w_qkv = weight((heads + 2 * kv_heads) * head_dim, width)
        self.w_out = weight(width, heads * head_dim)
        per = -(-max_tokens // page)  # pages a request may need
        pages, shape = batch * per, (batch * per, page, kv_heads, head_dim)
        kv = torch.int8 if q8 else dtype
        tensors = [torch.empty(shape, dtype=kv, device=device) for _ in range(2)]
        if q8:
            tensors += [torch.empty((*shape[:3], head_dim // 32), dtype=torch.float16, device=device) for _ in range(2)]
        self.cache = sdt.PagedCache(*tensors)
        self.workspace = sdt.paged_attn_workspace(heads, kv_heads, head_dim)
        # the pool of free pages, in the order in which they are handed out
        self.pool = torch.randperm(pages, generator=g, device=device).to(torch.int32)
        self.place = torch.zeros(2, dtype=torch.int32, device=device)  # ... and how many of them have been
        self.table = torch.full((batch, per), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.one_each = torch.ones(batch, dtype=torch.int32, device=device)  # a decode step's new tokens
        # the scheduler's own count of pages and tokens: no device read is needed
        self.taken, self.host_lens = 0, [0] * batch

    def project(self, x):
        """q, k and v of the rows of x, as slices of the fused projection's rows."""
        rows = sdt.gemm_ex(x, self.w_qkv.t())
        q, k, v = rows.unflatten(1, (-1, self.head_dim)).split((self.heads, self.kv_heads, self.kv_heads), dim=1)
        return q, k, v

    def enqueue_store(self, k, v, new):
        """Gives the requests' new tokens (a count each, on the GPU) pages and slots, and stores them, request after request."""
        slots = torch.empty(k.shape[0], dtype=torch.int64, device=k.device)
        sdt.paged_tables(self.lens, new, self.pool, self.table, page_size=self.page, slots=slots, kv_lens=self.lens, taken=self.place)
        sdt.paged_append(k, v, slots, self.cache)

    def enqueue_step(self, x):
        """A decode step's work on the GPU: the layer's output for one new row per request."""
        q, k, v = self.project(x)
        self.enqueue_store(k, v, self.one_each)
        o = sdt.paged_attn_m1(q, self.cache, self.table, self.lens, workspace=self.workspace)
        return sdt.gemm_ex(o.flatten(1), self.w_out.t())

    def count(self, new):
        """The scheduler's side of new[b] more tokens of request b."""
        for b, n in enumerate(new):
            self.taken += -(-(self.host_lens[b] + n) // self.page) - -(-self.host_lens[b] // self.page)
            self.host_lens[b] += n

    def store(self, k, v, new):
        """Stores prompts: new[b] tokens of request b, request after request."""
        self.enqueue_store(k, v, torch.tensor(new, dtype=torch.int32, device=k.device))
        self.count(new)

    def step(self, x):
        """One decode step: the layer's output for one new row per request."""
        self.count([1] * x.shape[0])
        return self.enqueue_step(x)

    def captured(self, x):
        """A function that runs one decode step on the rows then in x by replaying a captured one, and its output."""
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = self.enqueue_step(x)

        def replay():
            self.count([1] * x.shape[0])
            graph.replay()

        return replay, y


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--batch", type=int, default=16)
    p.add_argument("--prompt", type=int, default=1000, help="tokens of the longest prompt; the others are shorter")
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--kv-heads", type=int, default=32)
    p.add_argument("--q8", action="store_true")
    p.add_argument("--graph", action="store_true", help="capture one step and replay it")
    a = p.parse_args()
    layer = Layer(a.batch, a.prompt + a.steps, kv_heads=a.kv_heads, q8=a.q8)
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = [max(1, a.prompt - i * a.prompt // (2 * a.batch)) for i in range(a.batch)]
    _, k, v = layer.project(torch.randn(sum(prompts), 4096, generator=g, device="cuda").to(torch.bfloat16))
    layer.store(k, v, prompts)
    x = torch.randn(a.batch, 4096, generator=g, device="cuda").to(torch.bfloat16)
    x = layer.step(x)  # first step: warm-up
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    if a.graph:
        replay, y = layer.captured(x)
    begin.record()
    for _ in range(a.steps - 1):
        if a.graph:
            replay()
            x.copy_(y)
        else:
            x = layer.step(x)
    end.record()
    sdt.check_device_status()
    print(f"{a.batch} requests, {sum(layer.host_lens)} cached tokens, {layer.taken} pages of {layer.page}, "
          f"{'q8' if a.q8 else 'bf16'} cache: {begin.elapsed_time(end) * 1e3 / max(1, a.steps - 1):.1f} us a step; "
          f"|output| mean {x.float().abs().mean().item():.4f}")


if __name__ == "__main__":
    main()
