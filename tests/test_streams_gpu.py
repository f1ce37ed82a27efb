"""Outputs that the products allocate for a call on a stream that is not the current one: never memory that
another stream may still be using, before or after."""
import pytest
import torch

import shape_driven_tile_gb300 as sdt

pytestmark = pytest.mark.gpu
LONG = 30_000_000  # cycles that a stream is kept busy: some 15 ms


def calls(dev):
    g = torch.Generator(device=dev).manual_seed(0)
    a, b = (torch.randn(256, 512, generator=g, device=dev).half() for _ in range(2))
    b = b.t().contiguous()
    x, w = torch.randn(512, generator=g, device=dev).to(torch.bfloat16), torch.randn(640, 512, generator=g, device=dev).to(torch.bfloat16)
    q, s = torch.randint(-127, 128, (640, 512), generator=g, device=dev, dtype=torch.int8), torch.rand(640, 16, generator=g, device=dev).half()
    ws = sdt.gemm_workspace()
    return {"gemm_f16": lambda st: sdt.gemm_f16(a, b, stream=st), "gemm_ex": lambda st: sdt.gemm_ex(a, b, stream=st),
            "gemm_f16_ws": lambda st: sdt.gemm_f16_ws(a, b, workspace=ws, stream=st),
            "gemm_ex_ws": lambda st: sdt.gemm_ex_ws(a, b, workspace=ws, stream=st),
            "gemm_f16_with_tile": lambda st: sdt.gemm_f16_with_tile(a, b, tile=0, stream=st),
            "gemv_m1_bf16": lambda st: sdt.gemv_m1_bf16(x, w, stream=st), "gemv_m1_q8": lambda st: sdt.gemv_m1_q8(x, q, s, stream=st)}


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["gemm_f16", "gemm_ex", "gemm_f16_ws", "gemm_ex_ws", "gemm_f16_with_tile", "gemv_m1_bf16", "gemv_m1_q8"])
def test_outputs_of_a_call_on_another_stream(cuda_device, name, raw):
    call = calls(cuda_device)[name]
    want = call(None).clone()
    other = torch.cuda.Stream()
    stream = other.cuda_stream if raw else other
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    busy = torch.empty_like(want).data_ptr()  # freed, but the current stream may still be reading it
    got = call(stream)
    assert got.data_ptr() != busy
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    with torch.cuda.stream(other):
        torch.cuda._sleep(LONG)
    late = call(stream).data_ptr()  # freed before the other stream has written it
    assert torch.empty_like(want).data_ptr() != late
    torch.cuda.synchronize()
