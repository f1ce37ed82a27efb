"""A decode product right behind the product that writes its activations: launched while that one still
runs, it must read what that one writes and not what the buffer held before."""
import pytest
import torch

import shape_driven_tile_gb300 as sdt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("captured", [False, True])
def test_gemv_reads_the_activations_just_written(cuda_device, captured, q8):
    K, N, rounds = 2048, 1024, 12
    g = torch.Generator(device=cuda_device).manual_seed(5)
    bf16 = torch.bfloat16
    rows = torch.randn(rounds, 8, K, generator=g, device=cuda_device).to(bf16)
    w = (torch.randn(K, K, generator=g, device=cuda_device) * K ** -0.5).to(bf16)
    x = torch.zeros(8, K, dtype=bf16, device=cuda_device)
    a = torch.zeros(8, K, dtype=bf16, device=cuda_device)
    y = torch.zeros(N, dtype=torch.float32, device=cuda_device)
    if q8:
        weights = (torch.randint(-127, 128, (N, K), generator=g, device=cuda_device, dtype=torch.int8),
                   (torch.rand(N, K // 32, generator=g, device=cuda_device) * 0.01).half())
        product = sdt.gemv_m1_q8
    else:
        weights, product = ((torch.randn(N, K, generator=g, device=cuda_device)).to(bf16),), sdt.gemv_m1_bf16

    def step():
        product(x[0], *weights, y)  # also reads x before it is written again
        sdt.gemm_ex(a, w, x)
        product(x[0], *weights, y)

    run = step
    if captured:
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        run = graph.replay
    got = []
    for r in rows:
        a.copy_(r)
        run()
        got.append(y.clone())
    for r, have in zip(rows, got):
        want_x = sdt.gemm_ex(r, w)
        torch.cuda.synchronize()
        want = product(want_x[0].clone(), *weights)
        torch.cuda.synchronize()
        assert torch.equal(have, want)
    sdt.check_device_status()
