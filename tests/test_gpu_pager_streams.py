"""GPU tests of a pager used on other streams than the one it was created on."""
import pytest
import torch

import jagged_attention_gb300 as jfa

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    jfa.build()


def _pager():
    return jfa.Pager(max_seqs=2, max_pages=4, num_pages=8, page_size=16, H=8, Hkv=2, D=128)


def _cache():
    kp, vp = (torch.randn((8, 16, 2, 128), device="cuda").to(BF16) for _ in range(2))
    table = torch.arange(8, device="cuda", dtype=I32).view(2, 4)
    return kp, vp, table, torch.tensor([60, 33], device="cuda", dtype=I32), torch.randn((2, 8, 128), device="cuda").to(BF16)


def _busy(stream):
    """Some 0.3 s of work on the stream."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(600_000_000)


def _decode(pager, kp, vp, table, lens, q, stream):
    jfa.paged_decode(pager, q, kp, vp, table, lens, 0.1, stream=stream)


def _append(pager, kp, vp, table, lens, q, stream):
    jfa.paged_append(pager, kp[0, :2], vp[0, :2], lens, kp, vp, stream=stream)


def _tables(pager, kp, vp, table, lens, q, stream):
    jfa.paged_tables(pager, lens, table[0, :2], table, table.view(-1), lens[1:], rows=0, stream=stream)


@pytest.mark.parametrize("call", [_decode, _append, _tables])
@pytest.mark.parametrize("how", ["torch", "handle", "current"])
def test_a_dropped_pager_keeps_its_block_until_its_calls_are_done(call, how):
    """The block of a pager dropped while a call of another stream waits there is given to no other tensor before."""
    args = _cache()
    side = torch.cuda.Stream()
    call(_pager(), *args, None)  # the first call of a kind loads its kernel, which takes longer than _busy
    torch.cuda.synchronize()
    pager = _pager()
    at, size = pager.block.data_ptr(), pager.block.numel()
    _busy(side)
    if how == "current":
        with torch.cuda.stream(side):
            call(pager, *args, None)
    else:
        call(pager, *args, side if how == "torch" else side.cuda_stream)
    del pager
    others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not side.query()  # the call has not begun
    assert all(not at <= x.data_ptr() < at + size and not x.data_ptr() <= at < x.data_ptr() + size for x in others)
    side.synchronize()


def test_a_pager_is_cleared_when_it_is_there():
    """A call on any stream may follow at once: nothing of the creation is still to come."""
    args = _cache()
    made, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    _busy(made)
    with torch.cuda.stream(made):
        pager = _pager()
    assert made.query()
    _decode(pager, *args, side)
    assert pager.status(stream=side) == 0


def test_a_stream_that_captured_first_is_kept_track_of_all_the_same():
    """Work of a capture does not count: the first eager call behind it on the same stream does."""
    args = _cache()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    pager = _pager()
    out, lse = torch.empty_like(args[4]), torch.empty((8, 2), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        jfa.paged_decode(pager, args[4], *args[:2], *args[2:4], 0.1, out=out, lse=lse)
    graph.replay()
    torch.cuda.synchronize()
    at, size = pager.block.data_ptr(), pager.block.numel()
    _busy(side)
    _decode(pager, *args, side)
    del pager, graph
    others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not side.query()
    assert all(not at <= x.data_ptr() < at + size and not x.data_ptr() <= at < x.data_ptr() + size for x in others)
    side.synchronize()


def test_a_pager_made_within_a_capture():
    """Its clearing is the graph's, and nothing waits for the capturing stream."""
    args = _cache()
    want = jfa.paged_decode(_pager(), args[4], *args[:4], 0.1)
    out, lse = torch.empty_like(args[4]), torch.empty((8, 2), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pager = _pager()
        jfa.paged_decode(pager, args[4], *args[:2], *args[2:4], 0.1, out=out, lse=lse)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
