"""Eviction with every array in place, the lengths among them, as a captured decode loop calls it."""
import pytest
import torch

import evict_oracle as O
from routed_token_indexer_amd import _lib as M
from test_gpu_evict import caches, on

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lists", [1, 8])
@pytest.mark.parametrize("nseq,L,budget", [(3, 300, 100), (96, 600, 250), (5, 5000, 700), (2, 33000, 2000)])
def test_lengths_in_place(nseq, L, budget, lists):
    """new_len is lens: every list of a sequence goes by the old length, whichever ends first. More lists than the
    chip holds at once, so that some start when others have ended."""
    g = torch.Generator().manual_seed(L)
    k, _, t = caches(nseq, L, 50, 8, 8, seed=L, values=False)
    cap = t.shape[1] * 50
    mass = torch.rand(nseq, lists, cap, generator=g)
    lens = torch.tensor([L - 31 * (n % 7) for n in range(nseq)], dtype=torch.int32)
    lens[-1] = 10 ** 9                                   # clamped to what a sequence can address
    want = O.evict(mass, None, lens, budget, 2, 9)
    kc, tc, mc, lc = on(k), on(t), mass.cuda(), lens.cuda()
    pc = torch.arange(cap, dtype=torch.int32).expand(nseq, lists, cap).contiguous().cuda()
    pos = pc.clone()
    src = torch.empty(nseq, lists, budget, dtype=torch.int32, device="cuda")
    call = lambda: M.cache_evict(kc, None, mc, lc, budget, sinks=2, recent=9, pos=pc, table=tc, mass_out=mc,   # noqa: E731
                                 pos_out=pc, src=src, new_len=lc)
    moved = O.bits(O.move(k, want[1], t))

    def check():
        torch.cuda.synchronize()
        for x, y in zip((lc, src, mc, pc), want):
            assert torch.equal(x.cpu(), y)
        assert torch.equal(O.bits(kc), moved)
    assert call()[0] is lc
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for x, y in ((kc, k), (mc, mass), (lc, lens), (pc, pos)):
            x.copy_(y)
        graph.replay()
        check()
    # once more: what fits the budget stays as it is
    call()
    torch.cuda.synchronize()
    assert torch.equal(lc.cpu(), want[0]) and torch.equal(mc.cpu(), want[2]) and torch.equal(O.bits(kc), moved)
