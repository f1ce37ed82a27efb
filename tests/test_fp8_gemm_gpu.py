"""gemm_fp8 against the product in 64 bits: every tile, split and type, odd sizes, strides, values."""
import pytest
import torch

import shape_driven_tile_gb300 as sdt
from _fp8 import E4M3, E5M2, assert_near, fp8_values, product, scale_values

pytestmark = pytest.mark.gpu
TILES = [16, 32, 64, 128, 192, 256]


def operands(m, n, k, seed=0, at=E4M3, wt=E4M3):
    kb, nb = -(-k // 128), -(-n // 128)
    return (fp8_values((m, k), seed, at), scale_values((m, kb), seed + 1), fp8_values((n, k), seed + 2, wt),
            scale_values((nb, kb), seed + 3))


def check(a, sa, w, sw, out=None, **kw):
    got = sdt.gemm_fp8(a, sa, w, sw, out, **kw)
    sdt.check_device_status()
    want, slack = product(a, sa, w, sw)
    assert_near(got, want, slack)
    return got


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(1, 8, 16), (1, 128, 128), (3, 136, 144), (16, 256, 1024), (17, 248, 2000), (33, 1000, 640),
                                   (65, 128, 4112), (128, 384, 256), (129, 520, 1296), (300, 264, 400), (1000, 136, 272), (513, 2056, 1040)])
def test_sizes(cuda_device, m, n, k, out):
    check(*operands(m, n, k), out_dtype=out)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("splits", [1, 2, 3, 5, 8])
def test_tiles_and_splits(cuda_device, tile, splits):
    check(*operands(37, 392, 1808, seed=5), tile=tile, splits=splits)


@pytest.mark.parametrize("tile", TILES)
def test_many_blocks(cuda_device, tile):
    """More k-blocks than the ring has slots and the scales' buffers have places, several times."""
    check(*operands(20, 136, 24000, seed=6), tile=tile, splits=1, out_dtype=torch.float32)


@pytest.mark.parametrize("at", [E4M3, E5M2])
@pytest.mark.parametrize("wt", [E4M3, E5M2])
@pytest.mark.parametrize("m", [5, 200])
def test_types(cuda_device, at, wt, m):
    check(*operands(m, 264, 528, seed=7, at=at, wt=wt), out_dtype=torch.float32)


@pytest.mark.parametrize("m", [1, 16, 40, 129, 700])
def test_whole_numbers_are_exact(cuda_device, m):
    """Small whole numbers and scales that are powers of two: every sum is exact, in any order."""
    n, k = 272, 1040
    g = torch.Generator(device=cuda_device).manual_seed(m)
    a, w = (torch.randint(-8, 9, s, generator=g, device=cuda_device).float().to(E4M3) for s in ((m, k), (n, k)))
    sa, sw = (torch.exp2(torch.randint(-2, 3, s, generator=g, device=cuda_device).float()) for s in ((m, 9), (3, 9)))
    got = sdt.gemm_fp8(a, sa, w, sw, out_dtype=torch.float32)
    assert torch.equal(got.double(), product(a, sa, w, sw)[0])


@pytest.mark.parametrize("m", [7, 150])
def test_strides(cuda_device, m):
    """Padded rows, scales of either order and of a wider tensor, a column slice as output."""
    n, k = 200, 336
    a0, sa, w0, sw = operands(m, n, k + 48, seed=9)
    a, w = a0[:, 16:16 + k], w0[:, 32:32 + k]
    sa, sw = sa[:, :3].t().contiguous().t(), sw[:, :3].t().contiguous().t()
    rows = torch.full((m, n + 24), 7.0, dtype=torch.bfloat16, device=cuda_device)
    check(a, sa, w, sw, rows[:, 8:8 + n])
    assert (rows[:, :8] == 7).all() and (rows[:, 8 + n:] == 7).all()
    wide = torch.zeros((m, 9), device=cuda_device)
    wide[:, ::3] = sa
    check(a, wide[:, ::3], w, sw.contiguous(), out_dtype=torch.float16)
    one = scale_values((1, 1), 3)  # one scale for everything
    check(a, one.expand(m, 3), w, one.expand(2, 3))


def test_strides_of_single_rows_and_blocks_may_be_anything(cuda_device):
    a, sa, w, sw = operands(1, 72, 112, seed=10)
    far = 2 ** 33 + 5
    out = torch.zeros(72, dtype=torch.bfloat16, device=cuda_device).as_strided((1, 72), (far, 1))
    check(a.as_strided((1, 112), (far, 1)), sa.as_strided((1, 1), (far, far)), w, sw.as_strided((1, 1), (far, far)), out)
    x = torch.randn(1, 112, device=cuda_device).to(torch.bfloat16)
    q, s = sdt.quant_fp8(x)
    q1, s1 = (torch.zeros_like(t).as_strided(t.shape, (far, 1)) for t in (q, s))
    sdt.quant_fp8(x, q=q1, scales=s1.as_strided((1, 1), (far, far)))
    assert torch.equal(q1.float(), q.float()) and torch.equal(s1, s)


@pytest.mark.parametrize("m,n,k", [(0, 16, 32), (4, 0, 32), (4, 16, 0), (130, 264, 0)])
def test_empty(cuda_device, m, n, k):
    a, w = (torch.zeros(s, device=cuda_device).to(E4M3) for s in ((m, k), (n, k)))
    sa, sw = (torch.ones(s, device=cuda_device) for s in ((m, -(-k // 128)), (-(-n // 128), -(-k // 128))))
    got = sdt.gemm_fp8(a, sa, w, sw)
    assert got.shape == (m, n) and (got == 0).all()


@pytest.mark.parametrize("m", [1, 17, 200])
def test_nan_and_infinity_stay_in_their_rows(cuda_device, m):
    a, sa, w, sw = operands(m, 264, 400, seed=11)
    clean = sdt.gemm_fp8(a, sa, w, sw)
    row, col = m // 2, 130
    a2, sa2, w2 = a.clone(), sa.clone(), w.clone()
    a2.view(torch.uint8)[row, 399] = 0x7F  # NaN
    got = sdt.gemm_fp8(a2, sa, w, sw)
    assert got[row].isnan().all() and torch.equal(got[torch.arange(m) != row], clean[torch.arange(m) != row])
    w2.view(torch.uint8)[col, 0] = 0xFF
    got = sdt.gemm_fp8(a, sa, w2, sw)
    assert got[:, col].isnan().all() and torch.equal(got[:, torch.arange(264) != col], clean[:, torch.arange(264) != col])
    sa2[row, 1] = torch.inf
    got = sdt.gemm_fp8(a, sa2, w, sw)
    assert not got[row].isfinite().any() and torch.equal(got[torch.arange(m) != row], clean[torch.arange(m) != row])


@pytest.mark.parametrize("m", [1, 60, 500])
def test_the_same_call_gives_the_same_bits(cuda_device, m):
    ops = operands(m, 1032, 4000, seed=13)
    first = sdt.gemm_fp8(*ops, out_dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(sdt.gemm_fp8(*ops, out_dtype=torch.float32), first)


@pytest.mark.parametrize("m", [2, 400])
def test_captured_and_on_another_stream(cuda_device, m):
    a, sa, w, sw = operands(m, 512, 1024, seed=15)
    want = sdt.gemm_fp8(a, sa, w, sw)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = sdt.gemm_fp8(a, sa, w, sw, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    assert torch.equal(got, want)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(graph):
        sdt.gemm_fp8(a, sa, w, sw, out)
    a.copy_(a.flip(0).clone())
    sa.copy_(sa.flip(0).clone())
    graph.replay()
    assert torch.equal(out, want.flip(0))


@pytest.mark.parametrize("tile", [64, 128, 192, 256])
def test_outputs_past_32_bits(cuda_device, tile):
    """More than 2^31 results: the last rows and a few between."""
    m, n, k = 131088, 16400, 128
    a, sa, w, sw = operands(m, n, k, seed=17)
    got = sdt.gemm_fp8(a, sa, w, sw, tile=tile, splits=0 if tile > 128 else 1)
    sdt.check_device_status()
    at = torch.tensor([0, 1, 65535, 130943, 131000, m - 2, m - 1], device=cuda_device)
    want, slack = product(a[at], sa[at], w, sw)
    assert_near(got[at], want, slack)
    del got
    torch.cuda.empty_cache()


def test_both_kernels_side_by_side(cuda_device):
    """Calls on three streams at once, in every form, give what they give alone."""
    jobs = [(operands(m, n, k, seed=20 + i), tile) for i, (m, n, k, tile) in enumerate(
        [(1, 4096, 4096, 16), (700, 2048, 2048, 256), (40, 4096, 8192, 64), (100, 2048, 4096, 128), (3, 1024, 8192, 16)])]
    want = [sdt.gemm_fp8(*ops, tile=tile) for ops, tile in jobs]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for turn in range(40):
        for i, (ops, tile) in enumerate(jobs):
            with torch.cuda.stream(streams[(turn + i) % 3]):
                got.append((i, sdt.gemm_fp8(*ops, tile=tile)))
    torch.cuda.synchronize()
    assert all(torch.equal(t, want[i]) for i, t in got)
    sdt.check_device_status()
