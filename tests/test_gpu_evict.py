"""Eviction and moves against a plain sort: the same rows, the same bits, nothing else touched."""
import math

import pytest
import torch

import evict_oracle as O
from routed_token_indexer_amd import _lib as M

pytestmark = pytest.mark.gpu


def caches(nseq, L, page, heads, d, layout="token", dtype=torch.bfloat16, seed=0, table=True, values=True):
    g = torch.Generator().manual_seed(seed)
    cols = -(-L // page)
    r = lambda: torch.randint(-30000, 30000, (nseq * cols, heads, page, d) if layout == "head"   # noqa: E731
                              else (nseq * cols, page, heads, d), generator=g, dtype=torch.int16).view(dtype)
    k, v = r(), r() if values else None
    if layout == "head":
        k, v = k.permute(0, 2, 1, 3), None if v is None else v.permute(0, 2, 1, 3)
    t = torch.randperm(nseq * cols, generator=g).view(nseq, cols).to(torch.int32) if table else None
    return k, v, t


def on(x):
    if x is None:
        return None
    y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
    return y.copy_(x)


def both(k, v, t, mass, lens, budget, sinks=0, recent=0, pos=None, alias=False):
    kc, vc, tc, mc, lc = on(k), on(v), on(t), mass.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    pc = None if pos is None else pos.cuda()
    want = O.evict(mass, pos, torch.tensor(lens), budget, sinks, recent)
    got = M.cache_evict(kc, vc, mc, lc, budget, sinks=sinks, recent=recent, pos=pc, table=tc, mass_out=mc if alias else None,
                        pos_out=pc if alias else None)
    torch.cuda.synchronize()
    assert torch.equal(got[0].cpu(), want[0])
    assert torch.equal(got[1].cpu(), want[1])
    assert torch.equal(O.bits(got[2]), O.bits(want[2]))
    assert torch.equal(got[3].cpu(), want[3])
    for x, y in ((kc, k), (vc, v)):
        if y is not None:
            assert torch.equal(O.bits(x), O.bits(O.move(y, want[1], t)))
    return want


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("L,budget", [(1, 1), (2, 1), (63, 20), (64, 64), (65, 64), (300, 1), (300, 299), (1024, 100),
                                      (1025, 1000), (4096, 2000), (4097, 64)])
def test_lengths(L, budget, shared):
    g = torch.Generator().manual_seed(L + budget)
    heads = 2
    k, v, t = caches(3, L, 16, heads, 16, seed=L)
    cap = t.shape[1] * 16
    mass = torch.rand(3, 1 if shared else heads, cap, generator=g)
    lens = [L, max(0, L - 7), max(1, L // 2)]
    both(k, v, t, mass, lens, budget, sinks=min(budget // 4, 3), recent=min(budget // 2, 5), alias=L % 2 == 1)


@pytest.mark.parametrize("L", [16384, 16385, 49152, 49153, 70000])
def test_long_rows(L):
    """Rows whose keys stay in registers and longer ones, that are read again; in place and not."""
    g = torch.Generator().manual_seed(L)
    k, v, t = caches(1, L, 1000, 1, 8, seed=1)
    cap = t.shape[1] * 1000
    mass = torch.exp(2 * torch.randn(1, 1, cap, generator=g))
    pos = torch.randperm(cap, generator=g).view(1, 1, cap).to(torch.int32)
    for budget, alias in ((L // 3, True), (1000, False)):
        both(k, v, t, mass, [L], budget, sinks=4, recent=100, pos=pos, alias=alias)


@pytest.mark.parametrize("kind", ["equal", "few", "signs", "nan", "inf", "tiny", "near"])
@pytest.mark.parametrize("L,budget", [(200, 77), (3000, 1111), (20000, 5000)])
def test_ties_and_odd_masses(L, budget, kind):
    g = torch.Generator().manual_seed(budget)
    k, v, t = caches(2, L, 64, 1, 8, seed=2, values=False)
    cap = t.shape[1] * 64
    u = torch.rand(2, 1, cap, generator=g)
    mass = {"equal": torch.full_like(u, 0.25), "few": (u * 4).floor() / 4, "signs": torch.randn(2, 1, cap, generator=g).round(),
            "nan": torch.where(u < 0.3, torch.full_like(u, math.nan), u), "tiny": u * 2.0 ** -140,
            "inf": torch.where(u < 0.2, torch.full_like(u, math.inf), torch.where(u > 0.9, torch.full_like(u, -math.inf), u)),
            "near": 1.0 + (u * 300).floor() * 2.0 ** -23}[kind].clone()
    if kind == "signs":
        mass[mass == 0] = torch.where(torch.rand(int((mass == 0).sum()), generator=g) < 0.5, 0.0, -0.0)
    if kind == "nan":
        mass.view(torch.int32)[:, :, ::3] |= torch.where(mass[:, :, ::3].isnan(), -(1 << 31), 0).int()   # of both signs
    both(k, v, t, mass, [L, L - 3], budget, sinks=2, recent=9)


@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("d", [8, 24, 64, 96, 128, 256, 1024])
@pytest.mark.parametrize("heads,shared", [(1, True), (3, True), (3, False), (8, False)])
def test_rows_of_any_width(d, heads, shared, layout):
    g = torch.Generator().manual_seed(d)
    k, v, t = caches(2, 150, 24, heads, d, layout, torch.float16, seed=d, values=d != 24)
    mass = torch.rand(2, 1 if shared else heads, t.shape[1] * 24, generator=g)
    both(k, v, t, mass, [150, 131], 60, recent=10)


def test_lengths_out_of_range_and_missing_pages():
    k, v, t = caches(4, 100, 16, 2, 16, seed=4)
    t[0, 0], t[0, 6], t[1, 2] = -1, 10 ** 6, -3
    mass = torch.rand(4, 2, 112, generator=torch.Generator().manual_seed(1))
    both(k, v, t, mass, [100, 112, -5, 10 ** 6], 40, sinks=3, recent=8)
    both(k, v, t, mass, [0, 1, 40, 41], 40)
    both(k, v, t, mass, [100, 112, 50, 60], 500, sinks=3, recent=8)     # more than a sequence can hold


def test_positions():
    """Protection goes by position; equal and unordered positions, more protected ones than there is room for."""
    g = torch.Generator().manual_seed(9)
    k, v, t = caches(2, 128, 32, 2, 16, seed=5)
    mass = torch.rand(2, 2, 128, generator=g)
    pos = torch.randint(0, 100000, (2, 2, 128), generator=g, dtype=torch.int32)
    both(k, v, t, mass, [128, 90], 50, sinks=7, recent=40, pos=pos)
    both(k, v, t, mass, [128, 90], 50, sinks=7, recent=40, pos=torch.zeros_like(pos))
    both(k, v, t, mass, [128, 90], 50, sinks=0, recent=0, pos=pos)
    both(k, v, t, mass, [128, 90], 50, sinks=50, recent=0, pos=pos % 200)
    pos[0, 0, 5] = 2 ** 31 - 1
    both(k, v, t, mass, [128, 90], 50, sinks=1, recent=49, pos=pos)


@pytest.mark.parametrize("heads,shared", [(1, True), (4, False), (4, True)])
def test_another_cache_follows(heads, shared):
    g = torch.Generator().manual_seed(3)
    L, budget = 200, 70
    k, v, t = caches(3, L, 16, heads, 32, seed=6)
    mass = torch.rand(3, 1 if shared else heads, t.shape[1] * 16, generator=g)
    _, src, _, _ = O.evict(mass, None, torch.tensor([200, 90, 30]), budget, 2, 10)
    other = torch.randn(3, L, 128, generator=g).to(torch.bfloat16)       # index keys: one head, rows of whole sequences
    if shared:
        x = other.cuda()
        M.cache_move(x, None, src.cuda())
        assert torch.equal(O.bits(x), O.bits(O.move(other, src)))
    kc, vc = on(k), on(v)
    M.cache_move(kc, vc, src.cuda(), table=on(t))
    assert torch.equal(O.bits(kc), O.bits(O.move(k, src, t))) and torch.equal(O.bits(vc), O.bits(O.move(v, src, t)))
    # entries that are no rows, and lists longer than a sequence
    src = torch.full((3, src.shape[1], 300), -1, dtype=torch.int32)
    src[:, :, 3], src[:, :, 5], src[:, :, 7], src[:, :, 250] = 10 ** 6, 150, -9, 160
    kc = on(k)
    M.cache_move(kc, None, src.cuda(), table=on(t))
    assert torch.equal(O.bits(kc), O.bits(O.move(k, src, t)))
    M.cache_move(kc, None, src[:, :, :0].contiguous().cuda(), table=on(t))


def test_far_rows():
    """Rows behind 2^32 elements."""
    pages, page = 17000, 1024
    kc = torch.zeros(pages, page, 2, 128, dtype=torch.bfloat16, device="cuda")
    k, _, _ = caches(1, 2 * page, page, 2, 128, seed=7, values=False)
    at = [pages - 1, 8500]
    kc[at[0]], kc[at[1]] = k[0].cuda(), k[1].cuda()
    mass = torch.rand(1, 2, 2 * page, generator=torch.Generator().manual_seed(2))
    lens = torch.tensor([2 * page], dtype=torch.int32)
    got = M.cache_evict(kc, None, mass.cuda(), lens.cuda(), 900, table=torch.tensor([at], dtype=torch.int32).cuda())
    want = O.evict(mass, None, lens, 900, 0, 0)
    assert torch.equal(got[1].cpu(), want[1])
    moved = O.move(k, want[1], torch.tensor([[0, 1]], dtype=torch.int32))
    assert torch.equal(O.bits(kc[at[0]]), O.bits(moved[0])) and torch.equal(O.bits(kc[at[1]]), O.bits(moved[1]))


def test_graphs_and_streams():
    g = torch.Generator().manual_seed(10)
    k, v, t = caches(4, 500, 16, 2, 64, seed=8)
    mass, lens = torch.rand(4, 2, 512, generator=g).cuda(), torch.tensor([500, 400, 90, 500], dtype=torch.int32).cuda()
    want = O.evict(mass, None, lens, 100, 4, 20)
    kc, vc, tc = on(k), on(v), on(t)
    ws = torch.full((M.cache_workspace_bytes(M.OP_CACHE_EVICT, kc, tc, lists=2, budget=100),), 0xAB, dtype=torch.uint8,
                    device="cuda")
    outs = dict(mass_out=torch.empty_like(mass), pos_out=torch.empty(4, 2, 512, dtype=torch.int32, device="cuda"),
                src=torch.empty(4, 2, 100, dtype=torch.int32, device="cuda"),
                new_len=torch.empty(4, dtype=torch.int32, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        M.cache_evict(kc, vc, mass, lens, 100, sinks=4, recent=20, table=tc, ws=ws, **outs)
    for _ in range(3):
        kc.copy_(k)
        vc.copy_(v)
        for x in (*outs.values(), ws):
            x.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((outs["new_len"], outs["src"], outs["mass_out"], outs["pos_out"]), want):
            assert torch.equal(x.cpu(), y)
        assert torch.equal(O.bits(kc), O.bits(O.move(k, want[1], t))) and torch.equal(O.bits(vc), O.bits(O.move(v, want[1], t)))
    kc.copy_(k)
    side.wait_stream(torch.cuda.current_stream())
    got = M.cache_evict(kc, None, mass, lens, 100, sinks=4, recent=20, table=tc, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got[1].cpu(), want[1]) and torch.equal(O.bits(kc), O.bits(O.move(k, want[1], t)))


@pytest.mark.parametrize("L,budget,sinks,recent", [
    (700, 600, 300, 290),         # few rows left to rank, waves of protected ones, waves without rows
    (3000, 2900, 1000, 1500),
    (3000, 300, 200, 99),
    (9000, 8000, 4500, 3000),
    (20000, 15000, 9000, 5900),
    (40000, 39990, 25000, 14980),
    (40, 20, 0, 0),
    (520, 510, 512 - 40, 30),
])
@pytest.mark.parametrize("alias", [False, True])
def test_long_protected_runs(L, budget, sinks, recent, alias):
    g = torch.Generator().manual_seed(L)
    k, v, t = caches(2, L, 100, 1, 8, seed=3, values=False)
    mass = torch.rand(2, 1, t.shape[1] * 100, generator=g)
    both(k, v, t, mass, [L, L - 5], budget, sinks=sinks, recent=recent, alias=alias)


@pytest.mark.parametrize("L", [4096, 8192, 32768, 40000])
def test_every_row_moves(L):
    """Mass in the rows behind: the most moves there can be, more than workgroup memory lists; in a graph as well."""
    g = torch.Generator().manual_seed(L)
    k, v, t = caches(2, L, 64, 2, 8, seed=4, values=False)
    cap = t.shape[1] * 64
    mass = torch.rand(2, 2, cap, generator=g)
    mass[:, :, L // 2:] += 2
    both(k, v, t, mass, [L, L - 11], L // 2, alias=True)
    kc, tc = on(k), on(t)
    mc, lens = mass.cuda(), torch.tensor([L, L - 11], dtype=torch.int32, device="cuda")
    want = O.evict(mass, None, lens, L // 2, 0, 0)
    ws = torch.empty(M.cache_workspace_bytes(M.OP_CACHE_EVICT, kc, tc, lists=2, budget=L // 2), dtype=torch.uint8, device="cuda")
    src, new = torch.empty(2, 2, L // 2, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.cache_evict(kc, None, mc, lens, L // 2, table=tc, ws=ws, src=src, new_len=new, mass_out=mc)
    for _ in range(3):
        kc.copy_(k)
        mc.copy_(mass)
        ws.fill_(0x5A)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(src.cpu(), want[1]) and torch.equal(new.cpu(), want[0]) and torch.equal(mc.cpu(), want[2])
        assert torch.equal(O.bits(kc), O.bits(O.move(k, want[1], t)))


@pytest.mark.parametrize("L,budget", [(777, 300), (5001, 1000), (33001, 2000)])
def test_lists_that_start_anywhere(L, budget):
    """Lists of an odd number of rows, in arrays four bytes behind a 16-byte boundary."""
    g = torch.Generator().manual_seed(L)
    k, _, _ = caches(2, L, L, 3, 8, seed=5, table=False, values=False)
    mass, pos = torch.rand(2, 3, L, generator=g), torch.randperm(6 * L, generator=g).view(2, 3, L).to(torch.int32)

    def shifted(x):
        y = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape)
        return y.copy_(x)
    m, p, kc = shifted(mass), shifted(pos), on(k)
    lens = torch.tensor([L, L - 2], dtype=torch.int32)
    want = O.evict(mass, pos, lens, budget, 3, 50)
    got = M.cache_evict(kc, None, m, shifted(lens), budget, sinks=3, recent=50, pos=p, mass_out=m, pos_out=p,
                        src=shifted(torch.zeros(2, 3, budget, dtype=torch.int32)))
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x.cpu(), y)
    assert torch.equal(O.bits(kc), O.bits(O.move(k, want[1])))
