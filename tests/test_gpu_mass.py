"""Accumulated attention weight against the fp64 oracle: every head dimension, type, kind
of batch and layout; masks that leave rows or tokens empty; what is not seen."""
import math

import pytest
import torch

import evict_oracle as O
from routed_token_indexer_amd import _lib as M

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


class Batch:
    """nq queries for each sequence, the last ones of a cache of uneven lengths."""

    def __init__(self, d, dtype, nseq, nq, L, page, Hq, heads, layout="token", seed=0, table=True, big=1.0, spread=True):
        g = torch.Generator().manual_seed(seed)
        dt = TYPES[dtype]
        cols = -(-L // page)
        r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
        pages = nseq * cols
        k = r(pages, heads, page, d).permute(0, 2, 1, 3) if layout == "head" else r(pages, page, heads, d)
        self.kc = torch.empty_strided(k.shape, k.stride(), dtype=dt).copy_(k * big)
        self.vc = torch.empty_strided(k.shape, k.stride(), dtype=dt).copy_(r(*k.shape))
        self.table = torch.randperm(pages, generator=g).view(nseq, cols).to(torch.int32) if table else None
        self.lens = [max(nq, L - (n * L // (2 * nseq) if spread else 0)) for n in range(nseq)]
        fused = r(nseq * nq, Hq + 2, d).to(dt)
        self.q = fused[:, 1:1 + Hq]                                       # strided rows
        self.seq = torch.arange(nseq, dtype=torch.int32).repeat_interleave(nq)
        self.len = torch.tensor([self.lens[n] - nq + i + 1 for n in range(nseq) for i in range(nq)], dtype=torch.int32)
        self.nseq, self.heads, self.L, self.Hq = nseq, heads, cols * page, Hq

    def cuda(self):
        kc = torch.empty_strided(self.kc.shape, self.kc.stride(), dtype=self.kc.dtype, device="cuda").copy_(self.kc)
        return self, (self.q.cuda(), kc), (self.seq.cuda(), self.len.cuda()), None if self.table is None else self.table.cuda()


def both(b, lists=None, shuffle=None, lse=None, before=None, alias=False, **o):
    """Runs the call with the log-sums of the library's own attention, checks it, returns its sums."""
    if shuffle is not None:
        at = torch.randperm(len(b.seq), generator=torch.Generator().manual_seed(shuffle))
        b.q, b.seq, b.len = b.q[at], b.seq[at], b.len[at]
        o = {k: v[at] if k in ("q_start", "q_pos") else v for k, v in o.items()}
    b, (q, kc), (seq, ln), table = b.cuda()
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in o.items()}
    if lse is None:
        _, lse = M.attend(q, kc, _like(b, kc), seq, ln, table=table,
                          want_lse=True, **dev)
    G = lists or b.heads
    prior = None if before is None else before.cuda()
    out = prior if alias else torch.full((b.nseq, G, b.L), math.nan, device="cuda")
    got = M.attend_mass(q, kc, lse, seq, ln, table=table, mass=prior, out=out, **dev)
    assert got is out
    torch.cuda.synchronize()
    want = O.mass(b.q, b.kc, lse, b.seq, b.len, table=b.table, before=before, lists=G, **o)
    O.check_mass(got, want, f"{type(b).__name__}")
    return got, lse


def _like(b, kc):
    v = torch.empty_strided(kc.shape, kc.stride(), dtype=kc.dtype, device="cuda")
    return v.copy_(b.vc)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nq,heads,group,page,layout", [
    (1, 2, 4, 16, "token"),     # a decode step
    (1, 1, 16, 48, "head"),
    (1, 2, 17, 64, "token"),    # more than 16 rows
    (3, 2, 2, 1, "token"),      # pages of one token
    (40, 2, 3, 24, "head"),     # a window
    (97, 1, 8, 100, "token"),
])
def test_forms(d, dtype, nq, heads, group, page, layout):
    both(Batch(d, dtype, 2, nq, 300, page, heads * group, heads, layout, seed=d + nq))


@pytest.mark.parametrize("lists", [1, 4])
@pytest.mark.parametrize("nq", [1, 20])
@pytest.mark.parametrize("L", [1, 31, 32, 33, 127, 128, 129, 257])
def test_lengths(L, nq, lists):
    if nq > L:
        nq = L
    b = Batch(64, "bf16", 3, nq, L, 16, 8, 4, seed=L)
    both(b, lists=lists, before=torch.rand(3, lists, b.L), alias=L % 2 == 1)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nq", [1, 33])
@pytest.mark.parametrize("cap,bias", [(30.0, False), (5.0, True), (0.0, True), (1000.0, False), (0.5, False)])
def test_cap_and_bias(cap, bias, nq, d):
    b = Batch(d, "fp16", 2, nq, 200, 32, 6, 2, seed=nq + d, big=3.0)
    o = dict(cap=cap)
    if bias:
        o["slopes"] = 2.0 ** -torch.arange(1, 7, dtype=torch.float32)
        o["q_pos"] = b.len - 1 + 7
    both(b, **o)


@pytest.mark.parametrize("nq,group", [(1, 4), (60, 4)])
def test_intervals_in_any_order(nq, group):
    """Windows that start anywhere, empty ones, negative and excessive bounds; the queries shuffled."""
    b = Batch(128, "bf16", 3, nq, 333, 16, 2 * group, 2, seed=5)
    start = (b.len - 50).clone()
    start[0], b.len[-1] = 400, 10 ** 6
    if nq > 1:
        b.len[3], b.len[4], start[7], start[8] = 0, -5, -100, int(b.len[8])
        b.seq[9], b.seq[10] = 3, -1
    both(b, q_start=start, shuffle=3 if nq > 1 else None)
    both(Batch(128, "bf16", 3, nq, 333, 16, 2 * group, 2, seed=6), shuffle=4, lists=1)


def test_split_queries():
    """Long prompts over few keys, whose queries several workgroups share; a sequence of its own between them."""
    for lists in (1, 2):
        b = Batch(64, "bf16", 1, 1600, 1600, 64, 4, 2, seed=8)
        b.seq[500:520] = 7
        both(b, lists=lists)


def test_rows_without_weight_and_sums():
    """log-sums of -inf give nothing; otherwise the weights of a row sum to one."""
    b = Batch(128, "bf16", 2, 12, 150, 16, 8, 2, seed=11)
    got, lse = both(b)
    rows = torch.zeros(2, 2).index_add_(0, b.seq.long(), torch.full((24, 2), 4.0))
    assert bool(((got.sum(-1).cpu() - rows).abs() < 2e-5 * rows).all())
    lse = lse.clone()
    lse[3], lse[5, 2:] = -math.inf, -math.inf
    both(Batch(128, "bf16", 2, 12, 150, 16, 8, 2, seed=11), lse=lse)


@pytest.mark.parametrize("nq", [1, 30])
def test_unseen_may_hold_anything(nq):
    b = Batch(128, "bf16", 2, nq, 200, 16, 8, 2, seed=12)
    b.lens = [200, 200 - 50]
    first = 20
    start = torch.full_like(b.len, first)
    for n in range(2):
        for s in list(range(first)) + list(range(int(b.len[b.seq == n].max()), b.L)):
            b.kc[int(b.table[n, s // 16]), s % 16] = math.nan if s % 2 else math.inf
    got, _ = both(b, q_start=start)
    assert bool(got.isfinite().all()) and float(got[:, :, :first].abs().max()) == 0.0


@pytest.mark.parametrize("nq", [1, 30])
def test_missing_pages(nq):
    b = Batch(64, "fp16", 2, nq, 200, 16, 4, 2, seed=13)
    b.table[0, 3], b.table[1, 0], b.table[1, 5] = -1, 10 ** 6, -7
    got, _ = both(b)
    assert float(got[0, :, 48:64].abs().max()) == 0.0 and float(got[1, :, :16].abs().max()) == 0.0


def test_a_nan_reaches_what_it_touches():
    b = Batch(64, "bf16", 1, 25, 100, 16, 4, 2, seed=14)
    lse = torch.zeros(25, 4)
    b.kc[int(b.table[0, 2]), 5, 1] = math.nan                  # token 37 of kv head 1
    b.q = b.q.clone()
    b.q[20, 0] = math.nan                                      # a query head of kv head 0
    b, (q, kc), (seq, ln), table = b.cuda()
    got = M.attend_mass(q, kc, lse.cuda(), seq, ln, table=table).cpu()
    want = torch.zeros_like(got, dtype=torch.bool)
    want[0, 1, 37] = True
    want[0, 0, :int(b.len[20])] = True
    assert torch.equal(got.isnan(), want)


def test_rows_of_whole_sequences():
    for nq in (1, 20):
        b = Batch(128, "bf16", 3, nq, 64, 64, 8, 1, seed=15, table=False)
        both(b)
        b = Batch(128, "bf16", 3, nq, 64, 64, 8, 1, seed=15, table=False)
        _, lse = both(b)
        b, (q, kc), (seq, ln), _ = b.cuda()
        got = M.attend_mass(q, kc[:, :, 0], lse, seq, ln)
        O.check_mass(got, O.mass(b.q, b.kc, lse, b.seq, b.len))


@pytest.mark.parametrize("lists", [1, 2])
def test_no_queries(lists):
    kc = torch.randn(4, 16, 2, 64, device="cuda").to(torch.bfloat16)
    q = torch.empty(0, 4, 64, device="cuda", dtype=torch.bfloat16)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    before = torch.rand(4, lists, 16, device="cuda")
    got = M.attend_mass(q, kc, torch.empty(0, 4, device="cuda"), none, none, mass=before)
    assert torch.equal(got, before)
    assert float(M.attend_mass(q, kc, torch.empty(0, 4, device="cuda"), none, none, per_head=lists == 2).abs().max()) == 0.0


def test_far_rows():
    """Rows behind 2^32 bytes and behind 2^32 elements of the cache."""
    page, pages, heads, d = 1024, 17000, 2, 128
    kc = torch.empty(pages, page, heads, d, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[pages - 1, 9000]], dtype=torch.int32)
    b = Batch(d, "bf16", 1, 20, 2048, page, 4, heads, seed=16)
    kc[pages - 1], kc[9000] = b.kc[0].cuda(), b.kc[1].cuda()
    lse = torch.full((20, 4), 3.0)
    for nq in (20, 1):
        got = M.attend_mass(b.q[-nq:].cuda(), kc, lse[-nq:].cuda(), b.seq[-nq:].cuda(), b.len[-nq:].cuda(), table=table.cuda())
        want = O.mass(b.q[-nq:], b.kc, lse[-nq:], b.seq[-nq:], b.len[-nq:], table=torch.tensor([[0, 1]], dtype=torch.int32))
        O.check_mass(got, want)


@pytest.mark.parametrize("nq,lists", [(1, 2), (1, 1), (64, 2), (64, 1), (1200, 2)])
def test_graphs_and_repeats(nq, lists):
    """The same bits from run to run, also captured, with other work between the replays and on another stream."""
    b, (q, kc), (seq, ln), table = Batch(64, "bf16", 2, nq, max(nq, 300), 32, 8, 2, seed=17).cuda()
    lse = torch.full((2 * nq, 8), 4.0, device="cuda")
    before = torch.rand(2, lists, b.L, device="cuda")
    first = M.attend_mass(q, kc, lse, seq, ln, table=table, mass=before)
    out = torch.empty_like(first)
    need = M.cache_workspace_bytes(M.OP_ATTEND_MASS, kc, table, 2 * nq, 8, lists)
    ws = torch.full((max(need, 256),), 0xAB, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        M.attend_mass(q, kc, lse, seq, ln, table=table, mass=before, out=out, ws=ws)
    for _ in range(3):
        out.fill_(-1.0)
        ws.fill_(0xCD)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
        assert torch.equal(M.attend_mass(q, kc, lse, seq, ln, table=table, mass=before), first)
    q2 = q.clone()
    given = M.attend_mass(q2, kc, lse, seq, ln, table=table, mass=before, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(given, first)


@pytest.mark.parametrize("lists", [1, 2])
@pytest.mark.parametrize("d,nseq,nq,group", [(64, 70, 1, 4), (128, 40, 5, 3), (128, 9, 33, 2), (256, 5, 20, 4)])
def test_many_sequences(d, nseq, nq, group, lists):
    """Batches of uneven sequences, in order and with every sequence's queries spread over the batch."""
    for shuffle in (None, 7):
        b = Batch(d, "bf16", nseq, nq, 150, 16, 2 * group, 2, seed=nseq)
        both(b, lists=lists, shuffle=shuffle, before=torch.rand(nseq, lists, b.L, generator=torch.Generator().manual_seed(1)))


@pytest.mark.parametrize("nq", [1, 50])
def test_rows_far_apart(nq):
    """Queries whose rows lie more than 2^23 elements apart."""
    b = Batch(64, "bf16", 1, nq, 100, 16, 4, 2, seed=21)
    wide = torch.zeros(nq, (1 << 23) + 64, dtype=torch.bfloat16, device="cuda")
    q = wide[:, :256].view(nq, 4, 64)
    q.copy_(b.q)
    _, (_, kc), (seq, ln), table = b.cuda()
    _, lse = M.attend(q, kc, _like(b, kc), seq, ln, table=table, want_lse=True)
    got = M.attend_mass(q, kc, lse, seq, ln, table=table)
    assert torch.equal(lse, M.attend(q.contiguous(), kc, _like(b, kc), seq, ln, table=table, want_lse=True)[1])
    O.check_mass(got, O.mass(b.q, b.kc, lse, b.seq, b.len, table=b.table), "rows far apart")


def test_same_sums_every_time():
    """Split queries, a shared workspace, calls on two streams: the same bits."""
    b = Batch(128, "bf16", 2, 900, 900, 64, 8, 2, seed=22)
    _, (q, kc), (seq, ln), table = b.cuda()
    _, lse = M.attend(q, kc, _like(b, kc), seq, ln, table=table, want_lse=True)
    first = M.attend_mass(q, kc, lse, seq, ln, table=table)
    ws = torch.empty(max(256, M.cache_workspace_bytes(M.OP_ATTEND_MASS, kc, table, T=1800, Hq=8, lists=2)), dtype=torch.uint8,
                     device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(6):
        ws.fill_(255)
        assert torch.equal(M.attend_mass(q, kc, lse, seq, ln, table=table, ws=ws), first)
    got = [M.attend_mass(q, kc, lse, seq, ln, table=table, stream=streams[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, first) for x in got)


@pytest.mark.parametrize("nq,T", [(1, 0), (1, 3), (7, 0), (40, 0), (41, 0)])
def test_arrays_that_start_anywhere(nq, T):
    """Every array four bytes behind a 16-byte boundary, batches that are no multiple of four; sums as from aligned ones."""
    b = Batch(64, "bf16", 3, nq, 130, 10, 8, 2, seed=31)
    n = T or len(b.seq)
    _, (q, kc), (seq, ln), table = b.cuda()
    start = (ln - 60).clamp(min=0)
    _, lse = M.attend(q, kc, _like(b, kc), seq, ln, table=table, q_start=start, want_lse=True)

    def shifted(x):
        y = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape)
        return y.copy_(x)
    before = torch.rand(3, 2, b.L, device="cuda")
    want = M.attend_mass(q[:n], kc, lse[:n], seq[:n], ln[:n], table=table, q_start=start[:n], mass=before)
    got = M.attend_mass(q[:n], kc, shifted(lse[:n]), shifted(seq[:n]), shifted(ln[:n]), table=shifted(table),
                        q_start=shifted(start[:n]), mass=shifted(before), out=shifted(torch.empty_like(before)))
    assert torch.equal(got, want)
    O.check_mass(got, O.mass(b.q[:n], b.kc, lse[:n], b.seq[:n], b.len[:n], table=b.table, q_start=start[:n], before=before), "shifted")
