"""Accumulated weights of large head groups, positions left to the lengths, tables with more slots than sequences."""
import pytest
import torch

from test_gpu_mass import Batch, both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [31, 32, 33, 40, 63, 64, 65, 128, 130])
@pytest.mark.parametrize("nq,heads", [(1, 1), (3, 2), (21, 1)])
def test_large_groups(nq, heads, group, d):
    """Fewer heads than a step has rows, as many, and more, which take several steps a query."""
    both(Batch(d, "bf16", 2, nq, 150, 16, heads * group, heads, seed=d + group))


@pytest.mark.parametrize("d,group", [(64, 65), (128, 128), (256, 33)])
@pytest.mark.parametrize("lists", [1, 2])
def test_large_groups_of_split_queries(d, group, lists):
    """Enough rows that several workgroups share what sees a tile, some queries a sequence that there is not."""
    b = Batch(d, "fp16", 1, 120, 140, 20, 2 * group, 2, seed=d)
    b.seq[30:37] = 4
    both(b, lists=lists, shuffle=None if lists == 1 else 2)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nq", [1, 33])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_bias_by_lengths(cap, nq, d):
    """A distance bias without positions: a query stands at its last visible token."""
    b = Batch(d, "bf16", 2, nq, 200, 32, 6, 2, seed=nq + d, big=2.0)
    both(b, cap=cap, slopes=2.0 ** -torch.arange(1, 7, dtype=torch.float32))
    b = Batch(d, "bf16", 2, nq, 200, 32, 66, 1, seed=nq + d)
    both(b, cap=cap, slopes=torch.linspace(0.01, 0.5, 66), q_start=(b.len - 77).clamp(min=0))


@pytest.mark.parametrize("lists", [1, 2])
@pytest.mark.parametrize("nseq,nq", [(64, 33), (256, 64), (300, 8)])
def test_one_sequence_among_many_slots(nseq, nq, lists):
    """All queries of one sequence (and some of another) in a table of many."""
    b = Batch(64, "bf16", nseq, 1, 130, 16, 8, 2, seed=nseq, spread=False)
    g = torch.Generator().manual_seed(nq)
    b.q = torch.randn(nq + 3, 8, 64, generator=g).to(torch.bfloat16)
    b.seq = torch.full((nq + 3,), nseq // 2, dtype=torch.int32)
    b.seq[-3:] = nseq - 1
    b.len = torch.cat([torch.arange(130 - nq, 130), torch.tensor([130, 3, 77])]).int()
    both(b, lists=lists, before=torch.rand(nseq, lists, b.L, generator=g))
