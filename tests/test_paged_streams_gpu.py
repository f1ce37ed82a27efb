"""Outputs that paged_tables and paged_attn_m1 allocate for a call on a stream that is not the current one:
never memory that another stream may still be using, before or after."""
import pytest
import torch

import shape_driven_tile_gb300 as sdt

pytestmark = pytest.mark.gpu
LONG = 30_000_000  # cycles that a stream is kept busy: some 15 ms
B, H, D, PAGE, N = 512, 2, 64, 16, 20


def calls(dev):
    i32 = dict(dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev).manual_seed(0)
    kv = [torch.randn(64, PAGE, H, D, generator=g, device=dev).to(torch.bfloat16) for _ in range(2)]
    cache, ws = sdt.PagedCache(*kv), sdt.paged_attn_workspace(H, H, D)
    q = torch.randn(B, H, D, generator=g, device=dev).to(torch.bfloat16)
    table = torch.randint(0, 64, (B, 2), generator=g, **i32)
    lens, new, free = torch.full((B,), N, **i32), torch.ones(B, **i32), torch.arange(B, **i32)
    slots = torch.empty(B, dtype=torch.int64, device=dev)
    return {"attn": lambda s: (sdt.paged_attn_m1(q, cache, table, lens, workspace=ws, stream=s),),
            "tables": lambda s: sdt.paged_tables(lens, new, free, table.clone(), page_size=PAGE, slots=slots, stream=s)[:2]}


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["attn", "tables"])
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
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # blocks that the other stream has yet to write are not handed out to the current one
    with torch.cuda.stream(other):
        torch.cuda._sleep(LONG)
    got = call(stream)
    late = {t.data_ptr() for t in got}
    del got
    blocks = [torch.empty(s, dtype=d, device=cuda_device) for s, d in shapes]
    assert not late & {t.data_ptr() for t in blocks}
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["attn", "tables"])
def test_the_current_stream_by_its_handle(cuda_device, name):
    call = calls(cuda_device)[name]
    want = [t.clone() for t in call(None)]
    for stream in (torch.cuda.current_stream(), torch.cuda.current_stream().cuda_stream, 0):
        got = call(stream)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_what_the_caller_still_reads_is_not_written_again(cuda_device):
    """A result that the current stream is reading when its last reference goes is not handed to the other stream."""
    call, other = calls(cuda_device)["attn"], torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(other)[0]
    torch.cuda.current_stream().wait_stream(other)
    torch.cuda._sleep(LONG)
    kept, at = got.clone(), got.data_ptr()
    del got
    again = call(other)[0]
    assert again.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(kept, again)
