"""gemm_fp8's two-CTA tiles (and the widest one-CTA tile beside them) asked for by name: types, layouts of scales, strides,
non-finite values, capture, and pairs that run several tiles one after another."""
import pytest
import torch

import shape_driven_tile_gb300 as sdt
from _fp8 import E4M3, E5M2, assert_near, fp8_values, product, scale_values

pytestmark = pytest.mark.gpu
TILES = [128, 192, 256]


def operands(m, n, k, seed=0, at=E4M3, wt=E4M3, by_row=False):
    kb, nb = -(-k // 128), -(-n // 128)
    sa = scale_values((m, kb), seed + 1)
    if by_row:  # neighbouring rows' scales are neighbours
        sa = sa.t().contiguous().t()
    return fp8_values((m, k), seed, at), sa, fp8_values((n, k), seed + 2, wt), scale_values((nb, kb), seed + 3)


def check(a, sa, w, sw, out=None, **kw):
    got = sdt.gemm_fp8(a, sa, w, sw, out, **kw)
    sdt.check_device_status()
    want, slack = product(a, sa, w, sw)
    assert_near(got, want, slack)
    return got


def whole(m, n, k, seed, by_row):
    """Operands whose every sum is exact, in any order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    a, w = (torch.randint(-8, 9, s, generator=g, device="cuda").float().to(E4M3) for s in ((m, k), (n, k)))
    kb, nb = -(-k // 128), -(-n // 128)
    sa, sw = (torch.exp2(torch.randint(-2, 3, s, generator=g, device="cuda").float()) for s in ((m, kb), (nb, kb)))
    return a, sa.t().contiguous().t() if by_row else sa, w, sw


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("by_row", [False, True])
@pytest.mark.parametrize("at", [E4M3, E5M2])
@pytest.mark.parametrize("wt", [E4M3, E5M2])
def test_types_and_scale_layouts(cuda_device, tile, by_row, at, wt):
    for m, n, k in ((5, 136, 272), (300, 392, 1456)):
        check(*operands(m, n, k, seed=7, at=at, wt=wt, by_row=by_row), out_dtype=torch.float32, tile=tile)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("by_row", [False, True])
@pytest.mark.parametrize("m", [1, 129, 700])
def test_whole_numbers_are_exact(cuda_device, tile, by_row, m):
    ops = whole(m, 328, 1424, m, by_row)
    got = sdt.gemm_fp8(*ops, out_dtype=torch.float32, tile=tile)
    assert torch.equal(got.double(), product(*ops)[0])


# (tile, m, n, k): items of more than one round of this GPU's pairs of CTAs; on 152 SMs 76 whole tiles and 40 halves, 228 whole
# and 56 halves, 288 whole; 112 and 242 items.  The blocks of k are no multiple of the ring's slots or of the scales' buffers.
ROUNDS = [(256, 4096, 1288, 1424), (256, 4096, 4096, 656), (256, 8192, 2056, 832), (192, 4096, 1288, 1424), (192, 2816, 4104, 656),
          (128, 4096, 1288, 1424)]


@pytest.mark.parametrize("tile,m,n,k", ROUNDS)
@pytest.mark.parametrize("by_row", [False, True])
def test_several_tiles_one_after_another(cuda_device, tile, m, n, k, by_row):
    pairs = sdt.device_sm_count() // 2
    assert tile == 128 or -(-m // 256) * -(-n // tile) > pairs
    check(*operands(m, n, k, seed=31, by_row=by_row), tile=tile)
    ops = whole(m, n, k, 33, by_row)
    got = sdt.gemm_fp8(*ops, out_dtype=torch.float32, tile=tile)
    sdt.check_device_status()
    assert torch.equal(got.double(), product(*ops)[0])


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("tile", [192, 256])
def test_several_tiles_in_every_output_type(cuda_device, tile, out):
    check(*operands(4000, 1288, 912, seed=35), tile=tile, out_dtype=out)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("m", [7, 300])
def test_strides(cuda_device, tile, m):
    """Padded rows, scales of either order, stepped and expanded, a column slice as output."""
    n, k = 200, 336
    a0, sa, w0, sw = operands(m, n, k + 48, seed=9)
    a, w = a0[:, 16:16 + k], w0[:, 32:32 + k]
    sa, sw = sa[:, :3].t().contiguous().t(), sw[:, :3].t().contiguous().t()
    for dtype in (torch.bfloat16, torch.float32):
        rows = torch.full((m + 3, n + 24), 7.0, dtype=dtype, device=cuda_device)
        check(a, sa, w, sw, rows[:m, 8:8 + n], tile=tile)
        assert (rows[:, :8] == 7).all() and (rows[:, 8 + n:] == 7).all() and (rows[m:] == 7).all()
    wide = torch.zeros((m, 9), device=cuda_device)
    wide[:, ::3] = sa
    check(a, wide[:, ::3], w, sw.contiguous(), out_dtype=torch.float16, tile=tile)
    one = scale_values((1, 1), 3)  # one scale for everything
    check(a, one.expand(m, 3), w, one.expand(2, 3), tile=tile)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("m", [1, 200])
def test_nan_and_infinity_stay_in_their_rows(cuda_device, tile, m):
    a, sa, w, sw = operands(m, 264, 400, seed=11)
    clean = sdt.gemm_fp8(a, sa, w, sw, tile=tile)
    row, col = m // 2, 130
    a2, sa2, w2, others = a.clone(), sa.clone(), w.clone(), torch.arange(m, device=cuda_device) != row
    a2.view(torch.uint8)[row, 399] = 0x7F  # NaN
    got = sdt.gemm_fp8(a2, sa, w, sw, tile=tile)
    assert got[row].isnan().all() and torch.equal(got[others], clean[others])
    w2.view(torch.uint8)[col, 0] = 0xFF
    got, rest = sdt.gemm_fp8(a, sa, w2, sw, tile=tile), torch.arange(264, device=cuda_device) != col
    assert got[:, col].isnan().all() and torch.equal(got[:, rest], clean[:, rest])
    sa2[row, 1] = torch.inf
    got = sdt.gemm_fp8(a, sa2, w, sw, tile=tile)
    assert not got[row].isfinite().any() and torch.equal(got[others], clean[others])


@pytest.mark.parametrize("tile", TILES)
def test_the_same_call_gives_the_same_bits(cuda_device, tile):
    ops = operands(3000, 1032, 2000, seed=13)
    first = sdt.gemm_fp8(*ops, out_dtype=torch.float32, tile=tile)
    for _ in range(5):
        assert torch.equal(sdt.gemm_fp8(*ops, out_dtype=torch.float32, tile=tile), first)


@pytest.mark.parametrize("tile", TILES)
def test_captured_and_on_another_stream(cuda_device, tile):
    a, sa, w, sw = operands(3000, 1032, 656, seed=15)
    want = sdt.gemm_fp8(a, sa, w, sw, tile=tile)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = sdt.gemm_fp8(a, sa, w, sw, tile=tile, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    assert torch.equal(got, want)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(graph):
        sdt.gemm_fp8(a, sa, w, sw, out, tile=tile)
    a.copy_(a.flip(0).clone())
    sa.copy_(sa.flip(0).clone())
    graph.replay()
    assert torch.equal(out, want.flip(0))
