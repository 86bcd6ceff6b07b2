"""Calls that are given a stream of their own: what they make lies in that
stream's memory, and neither work queued on the current stream before the call
nor memory reused on it after the results are dropped meets theirs."""
import pytest
import torch

import attend_oracle as A
from routed_token_indexer_amd import _lib as M

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def home(x):
    """The stream from whose memory a tensor came."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= x.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    return None


def queue_work(a, b):
    """Some milliseconds of work on the current stream."""
    for _ in range(8):
        torch.mm(a, b, out=b)


@pytest.fixture(scope="module")
def big():
    return [torch.zeros(8192, 8192, dtype=BF, device="cuda") for _ in range(2)]


def attention(name):
    g = torch.Generator().manual_seed(3)
    kc, vc = (torch.randn(9, 64, 2, 128, generator=g).to(BF).cuda() for _ in range(2))
    q = torch.randn(4, 16, 128, generator=g).to(BF).cuda()
    seq = torch.arange(4, dtype=torch.int32, device="cuda")
    length = torch.tensor([64, 3, 30, 41], dtype=torch.int32, device="cuda")
    if name == "attend":
        f = lambda **kw: M.attend(q, kc, vc, seq, length, want_lse=True, **kw)  # noqa: E731
    elif name == "selected":
        idx = torch.randint(0, 64, (4, 50), generator=g).to(torch.int32).cuda()
        f = lambda **kw: M.attend_selected(q, kc, vc, idx, seq, length, want_lse=True, **kw)  # noqa: E731
    elif name == "shared":
        pre, plen = seq // 2 + 7, torch.full((9,), 60, dtype=torch.int32, device="cuda")
        f = lambda **kw: M.attend_shared(q, kc, vc, seq, length, pre, plen, want_lse=True, **kw)  # noqa: E731
    else:
        cs = torch.rand(64, 128, generator=g).cuda()
        tok = length - 1
        k, v = (torch.randn(4, 2, 128, generator=g).to(BF).cuda() for _ in range(2))
        f = lambda **kw: (M.cache_append(k, v, kc, vc, seq, tok, q=q, cos_sin=cs, **kw),)  # noqa: E731
    return f


@pytest.mark.parametrize("name", ["append", "attend", "selected", "shared"])
def test_a_stream_of_its_own(name, big):
    f = attention(name)
    want = f()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        # blocks of the outputs' and the workspace's sizes whose last work is still queued on the current stream
        queue_work(*big)
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 9, 1 << 12, 1 << 14, 1 << 16, 1 << 21, 1 << 25)
                for _ in range(2)]
        del junk
        got = f(stream=side)
        assert all(home(x) == side.cuda_stream for x in got)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        del got


def test_results_dropped_while_they_are_read(big):
    """A result goes back to its stream's memory only after the current stream's queued reads of it."""
    f = attention("attend")
    want = f()[0]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = f(stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    queue_work(*big)
    copy = out.clone()
    del out
    with torch.cuda.stream(side):
        other = [torch.full(want.shape, 7.0, dtype=BF, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(copy, want)
    del other


def test_an_indexer_on_a_stream_of_its_own(big):
    g = torch.Generator().manual_seed(8)
    q, k = torch.randn(4, 8, 128, generator=g).to(BF).cuda(), torch.randn(2, 512, 128, generator=g).to(BF).cuda()
    w = torch.rand(4, 8, generator=g).cuda()
    seq = torch.tensor([0, 0, 1, 1], dtype=torch.int32, device="cuda")
    length = torch.tensor([511, 512, 300, 301], dtype=torch.int32, device="cuda")
    kbar = M.pool_keys(k, 32)
    want = M.indexer(q, w, k, kbar, seq, length, 32, 4, 64)
    rows = M.debug_scores(q, w, k, None, seq, length)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    queue_work(*big)
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 9, 1 << 10, 1 << 13, 1 << 16, 1 << 21, 1 << 25)
            for _ in range(2)]
    del junk
    got = M.indexer(q, w, k, kbar, seq, length, 32, 4, 64, stream=side) + (
        M.debug_scores(q, w, k, None, seq, length, stream=side), M.pool_keys(k, 32, stream=side))
    assert all(home(x) == side.cuda_stream for x in got)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, (*want, rows, kbar)))


@pytest.mark.parametrize("name", ["append", "attend", "selected", "shared"])
def test_captured_on_a_stream_of_its_own(name, big):
    """A call given the capturing stream makes its outputs and workspace in the graph's memory: replays with work
    between them repeat the eager result."""
    f = attention(name)
    want = f()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = f(stream=side)
    for _ in range(4):
        for x in got:
            x.fill_(7)
        junk = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
        graph.replay()
        torch.mm(*big, out=big[1])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        del junk
