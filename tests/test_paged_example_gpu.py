"""The decode example: a step synchronises nothing, and a captured step replayed gives what steps give."""
import pytest
import torch

import shape_driven_tile_gb300 as sdt
from test_paged_decode_gpu import example

pytestmark = pytest.mark.gpu
PROMPTS, WIDTH = [16, 1, 33, 47, 15], 512


def layer(q8=False):
    made = example().Layer(len(PROMPTS), 80, width=WIDTH, heads=8, kv_heads=4, head_dim=64, page=16, q8=q8)
    g = torch.Generator(device="cuda").manual_seed(3)
    _, k, v = made.project(torch.randn(sum(PROMPTS), WIDTH, generator=g, device="cuda").to(torch.bfloat16))
    made.store(k, v, PROMPTS)
    return made, torch.randn(25, len(PROMPTS), WIDTH, generator=g, device="cuda").to(torch.bfloat16)


def test_a_step_does_not_synchronise(cuda_device):
    made, rows = layer()
    made.step(rows[0])
    torch.cuda.synchronize()
    was = torch.cuda.get_sync_debug_mode()
    torch.cuda.set_sync_debug_mode("error")
    try:
        for x in rows[1:4]:
            made.step(x)
    finally:
        torch.cuda.set_sync_debug_mode(was)
    sdt.check_device_status()


@pytest.mark.parametrize("q8", [False, True])
def test_a_captured_step(cuda_device, q8):
    a, rows = layer(q8)
    b, _ = layer(q8)
    want = [a.step(x).clone() for x in rows]
    x = rows[0].clone()
    got = [b.step(x).clone()]
    replay, y = b.captured(x)
    for r in rows[1:]:
        x.copy_(r)
        replay()
        got.append(y.clone())
    sdt.check_device_status()
    for s, t in zip(got, want):
        assert torch.equal(s, t)
    assert a.lens.tolist() == b.lens.tolist() == a.host_lens == b.host_lens == [n + len(rows) for n in PROMPTS]
    assert a.place.tolist() == b.place.tolist() == [a.taken, 0] and a.taken == b.taken
    assert torch.equal(a.table, b.table)


def test_example_runs_captured(cuda_device, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["paged_decode.py", "--batch", "3", "--prompt", "50", "--steps", "4", "--kv-heads", "8", "--graph"])
    example().main()
    assert "3 requests" in capsys.readouterr().out
