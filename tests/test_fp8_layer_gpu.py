"""The 8-bit operators together, as examples/fp8_layer.py runs them: each stage of a decode step against
64 bits on its actual inputs, captured steps, calls on several streams."""
import importlib.util
import os

import pytest
import torch

import shape_driven_tile_gb300 as sdt
from _fp8 import STEP, assert_near, assert_quantised, numbers, product

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMALL = dict(width=512, heads=4, kv_heads=2, head_dim=64, inner=640, page=8)


def example():
    spec = importlib.util.spec_from_file_location("fp8_layer", os.path.join(ROOT, "examples", "fp8_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def rows(n, width, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, width, generator=g, device="cuda").to(torch.bfloat16)


def filled(seed=0, prompts=(19, 1, 40), **kw):
    layer = example().Layer(len(prompts), max(prompts) + 6, seed=seed, **{**SMALL, **kw})
    layer.prompts(rows(sum(prompts), layer.norms[0].numel(), seed + 1), list(prompts))
    return layer


def norm64(r, w, eps=1e-6):
    v = r.double()
    return v * w.double() / torch.sqrt(v.square().mean(1, keepdim=True) + eps)


def test_each_stage_of_a_step(cuda_device):
    layer, batch = filled(), 3
    x, residual = rows(batch, 512, 5), 3 * rows(batch, 512, 6)
    positions = layer.lens.clone()
    assert positions.tolist() == [19, 1, 40]

    def normed(x, residual, w):
        want = (x.float() + residual.float()).to(torch.bfloat16)
        q, s = sdt.rms_norm_fp8(x, w, residual)
        assert torch.equal(residual, want)
        assert_quantised(q, s, norm64(want, w), (512 / 8 + 16) * 2.0 ** -24)
        return q, s

    def projected(q, s, w):
        out = sdt.gemm_fp8(q, s, *w)
        assert_near(out, *product(q, s, *w))
        return out

    qkv = projected(*normed(x, residual, layer.norms[0]), layer.w_qkv)
    q, k, v = qkv.unflatten(1, (-1, 64)).split((4, 2, 2), dim=1)
    angle = positions.double()[:, None] * torch.tensor(layer.rope.frequencies, dtype=torch.float64, device=cuda_device)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    want = []
    for t in (q, k):
        z = torch.complex(t[..., :32].double(), t[..., 32:].double()) * turn
        want.append(torch.cat([z.real, z.imag], 2))
    slack = 1e-6 * torch.cat([q, k], 1).double().abs().amax()  # 2^-25 turns and a few fp32 steps of the largest value
    sdt.rope_qk(q, k, positions, layer.rope, q_out=q, k_out=k)
    assert_near(q, want[0], slack)
    assert_near(k, want[1], slack)
    layer.store(k, v, layer.one_each)
    assert layer.lens.tolist() == [20, 2, 41]
    o = sdt.paged_attn_m1(q, layer.cache, layer.table, layer.lens, workspace=layer.workspace)
    for b, n in enumerate(layer.lens.tolist()):
        at = torch.arange(n, device=cuda_device)
        page = layer.table[b].long()[at // 8]
        kk, vv = (t[page, at % 8].double() for t in (layer.cache.k, layer.cache.v))
        assert torch.equal(kk[n - 1], k[b].double()) and torch.equal(vv[n - 1], v[b].double())
        for h in range(4):
            p = torch.softmax(kk[:, h // 2] @ q[b, h].double() / 8.0, 0)
            # softmax weights enter the product in 16 bits: half a step of each, and the output's rounding
            room = 2 * STEP[torch.bfloat16] * (p @ vv[:, h // 2].abs()) + 1e-6
            assert ((o[b, h].double() - p @ vv[:, h // 2]).abs() <= room).all()
    oq, os_ = sdt.quant_fp8(o.flatten(1))
    assert_quantised(oq, os_, o.flatten(1).double(), 0.0)
    y = projected(oq, os_, layer.w_out)
    both = projected(*normed(y, residual, layer.norms[1]), layer.w_gate_up)
    gate, up = both[:, :640], both[:, 640:]
    aq, as_ = sdt.quant_fp8(up, gate)
    assert_quantised(aq, as_, gate.double() * torch.sigmoid(gate.double()) * up.double(), 34 * 2.0 ** -22)
    out = projected(aq, as_, layer.w_down)
    # the same step as one call
    again = filled()
    residual2 = 3 * rows(batch, 512, 6)
    assert torch.equal(again.step(x, residual2), out) and torch.equal(residual2, residual)
    sdt.check_device_status()


def test_captured_steps_are_the_eager_ones(cuda_device):
    eager, graphed = filled(3), filled(3)
    x, r = rows(3, 512, 7), torch.zeros(3, 512, dtype=torch.bfloat16, device=cuda_device)
    xg, rg = x.clone(), r.clone()
    for layer, a, b in ((eager, x, r), (graphed, xg, rg)):
        a.copy_(layer.step(a, b))  # warm-up: the first call on a device may not be captured
    torch.cuda.synchronize()
    graph, y = graphed.captured(xg, rg)
    for _ in range(4):
        x = eager.step(x, r)
        graph.replay()
        xg.copy_(y)
        assert torch.equal(x, xg) and torch.equal(r, rg)
    assert torch.equal(eager.lens, graphed.lens)
    for b, n in enumerate(eager.lens.tolist()):  # (what lies behind a request's last token was never written)
        at = torch.arange(n, device=cuda_device)
        for name in ("k", "v"):
            held = [getattr(layer.cache, name)[layer.table[b].long()[at // 8], at % 8] for layer in (eager, graphed)]
            assert torch.equal(*held)
    sdt.check_device_status()


def test_layers_on_two_streams(cuda_device):
    """Two layers' steps at once, with the products' clusters side by side, change nothing."""
    alone = []
    for seed in (11, 12):
        layer, x, r = filled(seed, width=1024, inner=4096), rows(3, 1024, seed), torch.zeros(3, 1024, dtype=torch.bfloat16, device=cuda_device)
        alone.append([x := layer.step(x, r) for _ in range(5)] + [r])
    layers = [filled(seed, width=1024, inner=4096) for seed in (11, 12)]
    streams, got = [torch.cuda.Stream() for _ in layers], []
    torch.cuda.synchronize()
    state = [(rows(3, 1024, seed), torch.zeros(3, 1024, dtype=torch.bfloat16, device=cuda_device), []) for seed in (11, 12)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, (layer, stream) in enumerate(zip(layers, streams)):
            with torch.cuda.stream(stream):
                x, r, outs = state[i]
                x = layer.step(x, r)
                outs.append(x)
                state[i] = (x, r, outs)
    torch.cuda.synchronize()
    got = [s[2] + [s[1]] for s in state]
    for a, b in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    sdt.check_device_status()


def test_weights_of_the_example_are_near(cuda_device):
    w = torch.randn(200, 300, device=cuda_device)
    q, s = example().fp8_weight(w)
    assert q.shape == w.shape and s.shape == (2, 3)
    # half a step of e4m3 of each value, or of the smallest normal one of its block
    assert ((numbers(q, s, 128) - w.double()).abs() <= 2.0 ** -4 * w.double().abs() * 1.001 + 2.0 ** -10 * s.max()).all()


def test_the_example_runs(cuda_device, capsys, monkeypatch):
    for extra in ([], ["--graph"]):
        monkeypatch.setattr("sys.argv", ["fp8_layer.py", "--batch", "3", "--prompt", "20", "--steps", "3", "--inner", "512", *extra])
        example().main()
        assert "us a step" in capsys.readouterr().out
