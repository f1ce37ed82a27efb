"""Outputs that the 8-bit layer's operators allocate for a call on a stream that is not the current one: never
memory that another stream may still be using."""
import pytest
import torch

import shape_driven_tile_gb300 as sdt

pytestmark = pytest.mark.gpu
LONG = 30_000_000  # cycles that a stream is kept busy: some 15 ms


def calls(dev):
    g = torch.Generator(device=dev).manual_seed(0)
    x = torch.randn(700, 1024, generator=g, device=dev).to(torch.bfloat16)
    weight = torch.ones(1024, dtype=torch.bfloat16, device=dev)
    q, s = sdt.quant_fp8(x)
    sw = torch.ones(6, 8, device=dev)
    heads, positions, table = x.view(700, 8, 128), torch.arange(700, device=dev), sdt.RopeTable(128)
    return {"gemm": lambda st: (sdt.gemm_fp8(q, s, q[:696], sw, stream=st),),
            "quant": lambda st: sdt.quant_fp8(x, stream=st), "norm": lambda st: sdt.rms_norm_fp8(x, weight, stream=st),
            "rope": lambda st: sdt.rope_qk(heads, heads, positions, table, stream=st)}


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["gemm", "quant", "norm", "rope"])
def test_outputs_of_a_call_on_another_stream(cuda_device, name, raw):
    call = calls(cuda_device)[name]
    want = [t.clone() for t in call(None)]
    other = torch.cuda.Stream()
    stream = other.cuda_stream if raw else other
    torch.cuda.synchronize()
    shapes = [(t.shape, t.dtype) for t in want]
    # blocks that the current stream may still be reading are not written by the other one
    torch.cuda._sleep(LONG)
    blocks = [torch.empty(s, dtype=d, device=cuda_device) for s, d in shapes]
    busy = {t.data_ptr() for t in blocks}
    del blocks
    got = call(stream)
    assert not busy & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(torch.equal(a.float(), b.float()) for a, b in zip(got, want))
    # blocks that the other stream has yet to write are not handed out to the current one
    with torch.cuda.stream(other):
        torch.cuda._sleep(LONG)
    got = call(stream)
    late = {t.data_ptr() for t in got}
    del got
    blocks = [torch.empty(s, dtype=d, device=cuda_device) for s, d in shapes]
    assert not late & {t.data_ptr() for t in blocks}
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["gemm", "quant", "norm", "rope"])
def test_the_current_stream_by_its_handle(cuda_device, name):
    call = calls(cuda_device)[name]
    want = [t.clone() for t in call(None)]
    for stream in (torch.cuda.current_stream(), torch.cuda.current_stream().cuda_stream, 0):
        got = call(stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a.float(), b.float()) for a, b in zip(got, want))
