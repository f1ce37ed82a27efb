"""The decode example's layer, step by step, against the same layer in double precision with
the whole history of keys and values kept outside the cache."""
import importlib.util
import os

import pytest
import torch

import shape_driven_tile_gb300 as sdt

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_decode.py")


def example():
    spec = importlib.util.spec_from_file_location("paged_decode", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def q8(x):
    """Double values of x's q8 form (scale of 32 values fp16(max / 127))."""
    g = x.unflatten(-1, (-1, 32)).double()
    s = (g.abs().amax(-1, keepdim=True) * (1 / 127)).half().double()
    return (torch.round(g / s).clamp(-127, 127) * s).flatten(-2)


@pytest.mark.parametrize("kv_heads,quant", [(8, False), (2, False), (4, True)])
def test_steps_follow_the_reference(cuda_device, kv_heads, quant):
    heads, d, width, batch = 8, 64, 512, 5
    layer = example().Layer(batch, 60, width=width, heads=heads, kv_heads=kv_heads, head_dim=d, page=16, q8=quant)
    g = torch.Generator(device="cuda").manual_seed(3)
    keep = [([], []) for _ in range(batch)]  # every request's keys and values so far, as the projection gave them

    def remember(k, v, new):
        at = 0
        for b, n in enumerate(new):
            for store, t in zip(keep[b], (k, v)):
                store.append(t[at:at + n].clone())
            at += n

    prompts = [16, 1, 33, 47, 15]
    _, k, v = layer.project(torch.randn(sum(prompts), width, generator=g, device="cuda").to(torch.bfloat16))
    layer.store(k, v, prompts)
    remember(k, v, prompts)
    for _ in range(6):
        x = torch.randn(batch, width, generator=g, device="cuda").to(torch.bfloat16)
        y = layer.step(x)
        sdt.check_device_status()
        q, k, v = layer.project(x)
        remember(k, v, [1] * batch)
        o = torch.zeros(batch, heads, d, dtype=torch.float64, device="cuda")
        for b in range(batch):
            kk, vv = (torch.cat(t).double() if not quant else q8(torch.cat(t)) for t in keep[b])
            for h in range(heads):
                i = h * kv_heads // heads
                o[b, h] = torch.softmax(kk[:, i] @ q[b, h].double() * d ** -0.5, 0) @ vv[:, i]
        # attention output rounded to bf16 (2^-8 of it, both roundings of a near tie) goes through W; the sum of
        # 512 products in fp32 adds 512 * 2^-24 of sum |o w|; then the output's own rounding
        w = layer.w_out.double()
        want = o.flatten(1) @ w.t()
        tol = (2.0 ** -8 + 2.0 ** -12) * (o.flatten(1).abs() @ w.abs().t()) + 2.0 ** -8 * want.abs()
        assert ((y.double() - want).abs() <= tol).all()
    assert layer.lens.tolist() == layer.host_lens == [n + 6 for n in prompts]
    named = layer.table[layer.table >= 0]
    assert named.numel() == layer.taken and named.unique().numel() == layer.taken


def test_example_runs(cuda_device, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["paged_decode.py", "--batch", "3", "--prompt", "50", "--steps", "4", "--kv-heads", "8", "--q8"])
    example().main()
    assert "3 requests" in capsys.readouterr().out
