"""A decoder layer in 8 bits: prompts in, then one token a step, on the paged cache.

Each step runs, on one stream and without a synchronisation:

  rms_norm_fp8    the residual's addition and the norm, in fp8 with a scale per 128
  gemm_fp8        the fused q, k and v projection
  rope_qk         the new queries and keys to their positions, in place
  paged_tables, paged_append, paged_attn_m1   the cache (see paged_decode.py)
  quant_fp8       the attention's output in fp8
  gemm_fp8        the output projection
  rms_norm_fp8    again, with the residual
  gemm_fp8        both projections of the gated feed-forward block, side by side
  quant_fp8       silu(gate) * up in fp8
  gemm_fp8        back to the model's width

The default layer has the repository's decode benchmark's width (4096, 32 heads of 128).
Weights (fp8 with a scale per 128 x 128, made here from random 16-bit ones) and inputs are random.

    python examples/fp8_layer.py [--batch 16] [--prompt 1000] [--steps 32] [--kv-heads 8] [--inner 14336] [--graph]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import shape_driven_tile_gb300 as sdt  # noqa: E402


def fp8_weight(w):
    """w [N, K] as fp8 and float32 scales [ceil(N / 128), ceil(K / 128)], each block's largest value at 448."""
    n, k = w.shape
    blocks = torch.nn.functional.pad(w.float(), (0, -k % 128, 0, -n % 128)).unflatten(0, (-1, 128)).unflatten(2, (-1, 128))
    scales = blocks.abs().amax((1, 3)).clamp(min=2.0 ** -100) / 448.0
    q = (blocks / scales[:, None, :, None]).clamp(-448, 448).flatten(2).flatten(0, 1)[:n, :k]
    return q.to(torch.float8_e4m3fn).contiguous(), scales


class Layer:
    """One layer's weights, its pages and what it knows of its requests."""

    def __init__(self, batch, max_tokens, *, width=4096, heads=32, kv_heads=8, head_dim=128, inner=14336, page=16, seed=0,
                 device="cuda"):
        self.heads, self.kv_heads, self.head_dim, self.page, self.inner = heads, kv_heads, head_dim, page, inner
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, k):
            return fp8_weight(torch.randn(n, k, generator=g, device=device) * k ** -0.5)

        self.w_qkv = weight((heads + 2 * kv_heads) * head_dim, width)
        self.w_out = weight(width, heads * head_dim)
        self.w_gate_up = weight(2 * inner, width)
        self.w_down = weight(width, inner)
        self.norms = [(1.0 + 0.1 * torch.randn(width, generator=g, device=device)).to(torch.bfloat16) for _ in range(2)]
        self.rope = sdt.RopeTable(head_dim, device=device)
        per = -(-max_tokens // page)  # pages a request may need
        shape = (batch * per, page, kv_heads, head_dim)
        self.cache = sdt.PagedCache(*(torch.empty(shape, dtype=torch.bfloat16, device=device) for _ in range(2)))
        self.workspace = sdt.paged_attn_workspace(heads, kv_heads, head_dim)
        self.pool = torch.randperm(batch * per, generator=g, device=device).to(torch.int32)
        self.place = torch.zeros(2, dtype=torch.int32, device=device)
        self.table = torch.full((batch, per), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.one_each = torch.ones(batch, dtype=torch.int32, device=device)

    def project(self, x, residual, positions):
        """q, k and v of the rows of x + residual (which replaces residual), at their positions."""
        rows = sdt.gemm_fp8(*sdt.rms_norm_fp8(x, self.norms[0], residual), *self.w_qkv)
        q, k, v = rows.unflatten(1, (-1, self.head_dim)).split((self.heads, self.kv_heads, self.kv_heads), dim=1)
        sdt.rope_qk(q, k, positions, self.rope, q_out=q, k_out=k)
        return q, k, v

    def store(self, k, v, new):
        """Gives the requests' new tokens (a count each, on the GPU) pages and slots, and stores them, request after request."""
        slots = torch.empty(k.shape[0], dtype=torch.int64, device=k.device)
        sdt.paged_tables(self.lens, new, self.pool, self.table, page_size=self.page, slots=slots, kv_lens=self.lens, taken=self.place)
        sdt.paged_append(k, v, slots, self.cache)

    def prompts(self, x, new):
        """Stores prompts: new[b] rows of x for request b, request after request."""
        positions = torch.cat([torch.arange(n, device=x.device) for n in new])
        _, k, v = self.project(x, torch.zeros_like(x), positions)
        self.store(k, v, torch.tensor(new, dtype=torch.int32, device=x.device))

    def step(self, x, residual):
        """One decode step, one new row of x per request: the layer's output, which the next layer adds to the residual
        (updated in place)."""
        q, k, v = self.project(x, residual, self.lens)  # a new token's position is its request's length so far
        self.store(k, v, self.one_each)
        o = sdt.paged_attn_m1(q, self.cache, self.table, self.lens, workspace=self.workspace)
        y = sdt.gemm_fp8(*sdt.quant_fp8(o.flatten(1)), *self.w_out)
        both = sdt.gemm_fp8(*sdt.rms_norm_fp8(y, self.norms[1], residual), *self.w_gate_up)
        return sdt.gemm_fp8(*sdt.quant_fp8(both[:, self.inner:], both[:, :self.inner]), *self.w_down)

    def captured(self, x, residual):
        """A graph that replays one decode step on the rows then in x and residual, and its output."""
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = self.step(x, residual)
        return graph, y


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--batch", type=int, default=16)
    p.add_argument("--prompt", type=int, default=1000, help="tokens of the longest prompt; the others are shorter")
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--kv-heads", type=int, default=8)
    p.add_argument("--inner", type=int, default=14336)
    p.add_argument("--graph", action="store_true", help="capture one step and replay it")
    a = p.parse_args()
    if min(a.batch, a.prompt, a.steps) < 1:
        p.error("--batch, --prompt and --steps must be at least 1")
    layer = Layer(a.batch, a.prompt + a.steps, kv_heads=a.kv_heads, inner=a.inner)
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = [max(1, a.prompt - i * a.prompt // (2 * a.batch)) for i in range(a.batch)]
    layer.prompts(torch.randn(sum(prompts), 4096, generator=g, device="cuda").to(torch.bfloat16), prompts)
    x = torch.randn(a.batch, 4096, generator=g, device="cuda").to(torch.bfloat16)
    residual = torch.zeros_like(x)
    x = layer.step(x, residual)  # first step: warm-up
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    if a.graph:
        graph, y = layer.captured(x, residual)
    begin.record()
    for _ in range(a.steps - 1):
        if a.graph:
            graph.replay()
            x.copy_(y)
        else:
            x = layer.step(x, residual)
    end.record()
    sdt.check_device_status()
    print(f"{a.batch} requests, {sum(prompts) + a.batch * a.steps} cached tokens, fp8 layer of width 4096 and {a.inner}: "
          f"{begin.elapsed_time(end) * 1e3 / max(1, a.steps - 1):.1f} us a step; |output| mean {x.float().abs().mean().item():.4f}")


if __name__ == "__main__":
    main()
