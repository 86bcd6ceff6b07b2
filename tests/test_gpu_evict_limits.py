"""Eviction at the borders of its shapes and of positions."""
import pytest
import torch

from test_gpu_evict import both, caches

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L", [4095, 4096, 4097, 32767, 32768, 32769, 65600])
@pytest.mark.parametrize("fill", [1.0, 0.5, 0.03])
def test_rows_around_the_shapes(L, fill):
    """Rows that a sequence can address around 4096 and 32768, where the kernel changes its shape; full lists and lists
    of few tokens in long rows."""
    g = torch.Generator().manual_seed(L)
    k, v, t = caches(2, L, L, 2, 8, seed=1, table=False)
    mass = torch.exp(2 * torch.randn(2, 2, L, generator=g))
    pos = torch.randperm(4 * L, generator=g).view(2, 2, L).to(torch.int32)
    n = max(2, int(L * fill))
    for budget, alias in ((n // 2, True), (n - 1, False)):
        both(k, v, t, mass, [n, n - 1], budget, sinks=1, recent=budget // 3, pos=pos if alias else None, alias=alias)


@pytest.mark.parametrize("L,budget", [(90, 40), (6000, 500), (40000, 900)])
def test_positions_at_the_borders_of_32_bits(L, budget):
    g = torch.Generator().manual_seed(budget)
    k, v, t = caches(2, L, 100, 1, 8, seed=2, values=False)
    cap = t.shape[1] * 100
    mass = torch.rand(2, 1, cap, generator=g)
    low, high = -2 ** 31, 2 ** 31 - 1
    wide = torch.randint(low, high, (2, 1, cap), generator=g).to(torch.int32)
    ends = torch.where(torch.rand(2, 1, cap, generator=g) < 0.5, low, high).to(torch.int32)
    below = (low + torch.randint(0, 50, (2, 1, cap), generator=g)).to(torch.int32)
    above = (high - torch.randint(0, 50, (2, 1, cap), generator=g)).to(torch.int32)
    for pos in (wide, ends, below, above):
        for sinks, recent in ((0, 0), (0, budget), (budget, 0), (budget // 3, budget // 2)):
            both(k, v, t, mass, [L, L - 3], budget, sinks=sinks, recent=recent, pos=pos)
