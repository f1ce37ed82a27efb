"""paged_attn_m1 against the definition in double precision: types, head layouts, lengths,
page sizes, windows, strides; requests without keys; what lies outside the named tokens."""
import pytest
import torch

import _paged
import shape_driven_tile_gb300 as sdt

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def run(dev, lens, Hq, Hkv, D, page, dtype=BF16, q8=False, layout="token", window=0, scale=None, seed=0, spread=1.0, wide=None):
    table, pool = _paged.tables(lens, page, seed, wide=wide)
    cache = _paged.make_cache(pool, page, Hkv, D, dtype, layout, seed, q8)
    _paged.fill(cache, table, lens, seed + 1, dtype, spread)
    q = (torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(seed + 2)) * spread).to(dtype)
    on = [None if t is None else _to(t, dev) for t in cache]
    handle = sdt.PagedCache(*on)
    ws = sdt.paged_attn_workspace(Hq, Hkv, D)
    lse = torch.empty(len(lens), Hq, device=dev)
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    args = (q.to(dev), handle, table.to(dev), n)
    got = sdt.paged_attn_m1(*args, workspace=ws, window=window, scale=scale, lse=lse)
    sdt.check_device_status()
    want, want_lse, tol, tol_lse = _paged.attention(q, cache, table, lens, window, scale)
    _paged.assert_within(got, want, tol, "out")
    _paged.assert_within(lse, want_lse, tol_lse, "lse")
    assert not ws[: 1 << 20].any(), "counters left non-zero"
    again = sdt.paged_attn_m1(*args, workspace=ws, window=window, scale=scale)
    assert torch.equal(got.view(torch.int16), again.view(torch.int16)), "a second call differs"
    return got


def _to(t, dev):
    """The tensor on the device in the same order in memory."""
    return t.transpose(1, 2).to(dev).transpose(1, 2) if not t.is_contiguous() else t.to(dev)


EDGES = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 0]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_lengths_around_every_boundary(cuda_device, dtype, q8, D):
    run(cuda_device, EDGES, 8, 2, D, 16, dtype, q8)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("group", [1, 2, 5, 8, 9, 16, 17, 32, 33, 64, 70, 128])
def test_query_heads_per_key_head(cuda_device, group, q8):
    run(cuda_device, [0, 1, 77, 300], 2 * group, 2, 64, 16, BF16, q8, seed=group)


@pytest.mark.parametrize("group", [8, 24, 40])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("q8", [False, True])
def test_wide_heads_in_groups(cuda_device, group, D, q8):
    run(cuda_device, [5, 0, 513, 200], group, 1, D, 32, F16, q8, seed=group + D)


@pytest.mark.parametrize("D", [8, 24, 40, 72, 80, 96, 112, 136, 192, 224, 248])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_odd_head_widths(cuda_device, D, dtype):
    run(cuda_device, [1, 40, 130, 0, 99], 6, 3, D, 16, dtype, seed=D)


def test_q8_of_192_wide_heads(cuda_device):
    run(cuda_device, [1, 40, 130, 0, 99], 6, 3, 192, 16, BF16, True)


@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("page", [1, 3, 7, 16, 20, 64, 100, 256])
@pytest.mark.parametrize("q8", [False, True])
def test_page_sizes(cuda_device, page, layout, q8):
    run(cuda_device, [1, 50, 129, 400], 4, 2, 64, page, BF16, q8, layout, seed=page)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 399, 400, 401, 2 ** 31 - 1, 2 ** 40])
def test_sliding_window(cuda_device, window):
    run(cuda_device, [0, 1, 50, 129, 400], 4, 2, 64, 20, BF16, window=window)


@pytest.mark.parametrize("Hq,Hkv,D,q8", [(8, 1, 128, False), (32, 1, 64, False), (64, 1, 64, True), (4, 4, 128, True), (2, 1, 256, False)])
def test_one_long_request_split_over_the_grid(cuda_device, Hq, Hkv, D, q8):
    run(cuda_device, [20011], Hq, Hkv, D, 16, BF16, q8)


def test_mixed_lengths_share_the_grid(cuda_device):
    lens = [3000 if i % 7 == 0 else (i * 37) % 200 for i in range(150)]
    run(cuda_device, lens, 2, 2, 64, 16, F16)


def test_more_requests_than_threads(cuda_device):
    run(cuda_device, [(i * 13) % 40 for i in range(700)], 1, 1, 64, 16, BF16)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_peaked_scores_and_given_scale(cuda_device, dtype):
    run(cuda_device, [700, 33], 4, 1, 64, 16, dtype, spread=4.0, scale=0.3)
    run(cuda_device, [700, 33], 4, 1, 64, 16, dtype, scale=-0.7)
    run(cuda_device, [700, 33], 4, 1, 64, 16, dtype, scale=0.0)


def test_growing_scores_move_the_maximum(cuda_device):
    """Keys whose scores rise with their place: the running maximum moves in every unit."""
    n, D, page = 1500, 64, 16
    table, pool = _paged.tables([n], page, 0)
    cache = _paged.make_cache(pool, page, 1, D, F16, "token", 0)
    _paged.fill(cache, table, [n], 1, F16)
    pos = torch.arange(n)
    cache[0][table[0].long()[pos // page], pos % page, 0, 0] = (pos * 0.05).half()
    q = torch.ones(1, 2, D, dtype=F16)
    got = sdt.paged_attn_m1(q.cuda(), sdt.PagedCache(*[t.cuda() for t in cache[:2]]), table.cuda(),
                            torch.tensor([n], dtype=torch.int32).cuda(), workspace=sdt.paged_attn_workspace(2, 1, D), scale=1.0)
    want, _, tol, _ = _paged.attention(q, cache, table, [n], scale=1.0)
    _paged.assert_within(got, want, tol)


def test_all_requests_empty_and_no_requests(cuda_device):
    out = run(cuda_device, [0, 0, 0], 4, 2, 64, 16, wide=0)
    assert not out.any()
    q = torch.empty(0, 4, 64, dtype=BF16, device=cuda_device)
    cache = sdt.PagedCache(*[torch.zeros(1, 16, 2, 64, dtype=BF16, device=cuda_device) for _ in range(2)])
    e = torch.empty(0, dtype=torch.int32, device=cuda_device)
    assert sdt.paged_attn_m1(q, cache, e.view(0, 1), e, workspace=sdt.paged_attn_workspace(4, 2, 64)).shape == (0, 4, 64)


def test_infinite_scores(cuda_device):
    """A key that scores -inf has weight 0; a request whose keys all do gets zeros, as one without keys."""
    D = 64
    k = torch.zeros(2, 16, 1, D, dtype=BF16, device=cuda_device)
    v = torch.randn(2, 16, 1, D, device=cuda_device).to(BF16)
    k[0, :3, 0, 0] = -float("inf")
    k[1, :, 0, 0] = -float("inf")
    q = torch.zeros(2, 1, D, dtype=BF16, device=cuda_device)
    q[:, :, 0] = 1
    lse = torch.empty(2, 1, device=cuda_device)
    got = sdt.paged_attn_m1(q, sdt.PagedCache(k, v), torch.tensor([[0], [1]], dtype=torch.int32, device=cuda_device),
                            torch.tensor([5, 7], dtype=torch.int32, device=cuda_device),
                            workspace=sdt.paged_attn_workspace(1, 1, D), lse=lse)
    mean = v[0, 3:5, 0].double().mean(0).cpu()
    _paged.assert_within(got[0, 0], mean, 2.0 ** -8 * mean.abs() + 2.0 ** -14)
    assert not got[1].any() and lse[1, 0] == -float("inf")


def test_strided_operands(cuda_device):
    """q as a slice of fused projection rows, out and table as slices, keys and values in one tensor."""
    B, Hq, Hkv, D, page, lens = 5, 8, 2, 64, 16, [3, 0, 70, 200, 31]
    table, pool = _paged.tables(lens, page, 3)
    both = torch.full((pool, 2, page, Hkv, D), float("nan"), dtype=BF16)
    cache = (both[:, 0], both[:, 1], None, None)
    _paged.fill(cache, table, lens, 4, BF16)
    rows = torch.randn(B, (Hq + 2 * Hkv) * D, generator=torch.Generator().manual_seed(5)).to(BF16)
    q = rows[:, :Hq * D].unflatten(1, (Hq, D))
    on = both.to(cuda_device)
    wide_table = torch.full((B, table.shape[1] + 5), 10 ** 6, dtype=torch.int32, device=cuda_device)
    wide_table[:, :table.shape[1]] = table.to(cuda_device)
    out = torch.full((B, Hq, 2, D), 7.0, dtype=BF16, device=cuda_device)
    sdt.paged_attn_m1(rows.to(cuda_device)[:, :Hq * D].unflatten(1, (Hq, D)), sdt.PagedCache(on[:, 0], on[:, 1]),
                      wide_table[:, :table.shape[1]], torch.tensor(lens, dtype=torch.int32, device=cuda_device), out[:, :, 1],
                      workspace=sdt.paged_attn_workspace(Hq, Hkv, D))
    sdt.check_device_status()
    want, _, tol, _ = _paged.attention(q, cache, table, lens)
    _paged.assert_within(out[:, :, 1], want, tol)
    assert (out[:, :, 0] == 7.0).all()


def test_offsets_past_32_bits(cuda_device):
    """Pages whose elements lie more than 2^32 apart."""
    D, page, step = 64, 16, (1 << 32) + 64 * 64
    pool = torch.empty(step + page * D, dtype=BF16, device=cuda_device)
    k = torch.as_strided(pool, (2, page, 1, D), (step, D, D, 1))
    k.copy_(torch.randn(2, page, 1, D, generator=torch.Generator().manual_seed(0)).to(BF16))
    q = torch.randn(1, 4, D, generator=torch.Generator().manual_seed(1)).to(BF16)
    table, lens = torch.tensor([[1, 0]], dtype=torch.int32), [30]
    cache = sdt.PagedCache(k, k)
    got = sdt.paged_attn_m1(q.to(cuda_device), cache, table.to(cuda_device), torch.tensor(lens, dtype=torch.int32, device=cuda_device),
                            workspace=sdt.paged_attn_workspace(4, 1, D))
    want, _, tol, _ = _paged.attention(q, (k.cpu(), k.cpu(), None, None), table, lens)
    _paged.assert_within(got, want, tol)
    x = torch.randn(1, 1, D, generator=torch.Generator().manual_seed(2)).to(BF16).to(cuda_device)
    sdt.paged_append(x, x, torch.tensor([page + 3], device=cuda_device), cache)
    assert torch.equal(k[1, 3, 0], x[0, 0])


def test_bad_pages_and_lengths_are_reported_and_not_followed(cuda_device):
    D, dev = 64, cuda_device
    k = torch.ones(4, 16, 1, D, dtype=BF16, device=dev)
    cache, ws = sdt.PagedCache(k, k), sdt.paged_attn_workspace(2, 1, D)
    q = torch.ones(2, 2, D, dtype=BF16, device=dev)
    good = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=dev)
    for bad in (4, -1, 2 ** 31 - 1, -2 ** 31):
        table = good.clone()
        table[1, 1] = bad
        sdt.paged_attn_m1(q, cache, table, torch.tensor([20, 20], dtype=torch.int32, device=dev), workspace=ws)
        with pytest.raises(sdt.SdtError) as e:
            sdt.check_device_status()
        assert e.value.status == "SDT_ERR_ARG" and "page" in str(e.value)
        # the entry is not read where the length does not reach it
        sdt.paged_attn_m1(q, cache, table, torch.tensor([20, 16], dtype=torch.int32, device=dev), workspace=ws)
        sdt.check_device_status()
    out = sdt.paged_attn_m1(q, cache, good, torch.tensor([33, -5], dtype=torch.int32, device=dev), workspace=ws)
    with pytest.raises(sdt.SdtError, match="length"):
        sdt.check_device_status()
    assert (out[0] == 1).all() and not out[1].any()


def test_other_stream_and_shared_workspace(cuda_device):
    """Two calls in a row on a stream of their own, sharing a workspace with each other."""
    dev, D, page = cuda_device, 128, 16
    lens = [5000, 300]
    table, pool = _paged.tables(lens, page, 1)
    cache = _paged.make_cache(pool, page, 2, D, F16, "token", 0)
    _paged.fill(cache, table, lens, 2, F16)
    q = torch.randn(2, 8, D, generator=torch.Generator().manual_seed(3)).to(F16)
    handle, ws = sdt.PagedCache(*[t.to(dev) for t in cache[:2]]), sdt.paged_attn_workspace(8, 2, D)
    want, _, tol, _ = _paged.attention(q, cache, table, lens)
    on = (q.to(dev), handle, table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        outs = [sdt.paged_attn_m1(*on, workspace=ws) for _ in range(5)]
    given = torch.empty_like(outs[0])
    stream.synchronize()
    sdt.paged_attn_m1(*on, given, workspace=ws, stream=stream)
    stream.synchronize()
    for o in [*outs, given]:
        _paged.assert_within(o, want, tol)


def test_graph_replay_follows_the_lengths(cuda_device):
    """One captured call serves steps of other lengths: nothing on the host depends on them."""
    dev, D, page = cuda_device, 64, 16
    lens = [900, 40, 333]
    table, pool = _paged.tables(lens, page, 1)
    cache = _paged.make_cache(pool, page, 2, D, BF16, "token", 0)
    _paged.fill(cache, table, lens, 2, BF16)
    q = torch.randn(3, 4, D, generator=torch.Generator().manual_seed(3)).to(BF16)
    handle, ws = sdt.PagedCache(*[t.to(dev) for t in cache[:2]]), sdt.paged_attn_workspace(4, 2, D)
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    qd, td, out = q.to(dev), table.to(dev), torch.empty(3, 4, D, dtype=BF16, device=dev)
    sdt.paged_attn_m1(qd, handle, td, n, out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sdt.paged_attn_m1(qd, handle, td, n, out, workspace=ws)
    for step in ([900, 40, 333], [1, 0, 17], [64, 40, 128]):
        n.copy_(torch.tensor(step, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want, _, tol, _ = _paged.attention(q, cache, table, step)
        _paged.assert_within(out, want, tol)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,heads,q8", [(64, 8, False), (128, 8, False), (256, 4, False), (64, 8, True), (128, 8, True), (256, 4, True),
                                        (40, 8, False), (192, 4, True)])
def test_many_items(cuda_device, D, heads, q8, dtype):
    """Enough requests and heads for CTAs of one warp (and, in q8 of 128, of four all the same)."""
    lens = [(i * 29) % 70 for i in range(256)]
    lens[100], lens[255] = 1500, 600
    run(cuda_device, lens, 2 * heads, heads, D, 16, dtype, q8, layout="head", seed=D)


def test_many_items_of_odd_pages_in_a_window(cuda_device):
    lens = [(i * 31) % 150 for i in range(240)]
    run(cuda_device, lens, 16, 8, 64, 12, BF16, window=77)
    run(cuda_device, lens, 56, 8, 80, 12, F16, window=77)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("group,D", [(8, 128), (16, 128), (32, 128), (64, 128), (40, 64), (64, 64), (12, 256), (30, 256), (64, 256), (70, 256)])
def test_many_pieces_of_an_item(cuda_device, group, D, q8):
    """Few long requests of one key head: more pieces than one CTA joins at once, or pieces so large that a
    kernel of its own joins them."""
    run(cuda_device, [30007, 5, 0, 2049], group, 1, D, 16, BF16, q8, seed=group)


def test_steps_that_split_otherwise_share_a_workspace(cuda_device):
    """One workspace for calls that join in the kernel, in a second kernel, and not at all."""
    dev = cuda_device
    ws = sdt.paged_attn_workspace(64, 1, 256)
    for D, group, lens in ((256, 64, [9000]), (128, 8, [9000]), (128, 64, [20, 1]), (256, 64, [700, 800, 10]), (256, 64, [9000])):
        table, pool = _paged.tables(lens, 16, 3)
        cache = _paged.make_cache(pool, 16, 1, D, F16, "token", 0)
        _paged.fill(cache, table, lens, 4, F16)
        q = torch.randn(len(lens), group, D, generator=torch.Generator().manual_seed(5)).to(F16)
        got = sdt.paged_attn_m1(q.to(dev), sdt.PagedCache(*[t.to(dev) for t in cache[:2]]), table.to(dev),
                                torch.tensor(lens, dtype=torch.int32, device=dev), workspace=ws)
        want, _, tol, _ = _paged.attention(q, cache, table, lens)
        _paged.assert_within(got, want, tol)
        assert not ws[: 1 << 20].any()
