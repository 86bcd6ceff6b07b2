"""The attention operators against their plain forms in fp64: misa_attend,
misa_attend_selected and misa_attend_shared over paged and row caches, at the
sizes, masks and layouts where tiles, pages and parts end."""
import math

import pytest
import torch

import attend_oracle as A
from routed_token_indexer_amd import _lib as M

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def cache(g, nseq, cols, page, heads, d, dtype, layout="token", spare=2, paged=True):
    """k, v [pages, page, heads, d] and a table with the pages in any order.
    Pages outside the table hold NaN."""
    npages = nseq * cols + (spare if paged else 0)
    table = torch.randperm(npages, generator=g)[:nseq * cols].view(nseq, cols).to(torch.int32) if paged else None
    out = []
    for _ in range(2):
        x = torch.randn(npages, page, heads, d, generator=g)
        if paged:
            unused = torch.ones(npages, dtype=torch.bool)
            unused[table.flatten().long()] = False
            x[unused] = math.nan
        x = x.to(dtype).cuda()
        if layout == "head":
            x = x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
        out.append(x)
    return out[0], out[1], table.cuda() if paged else None


def ints(v):
    return torch.as_tensor(v, dtype=torch.int32).cuda()


def poison_behind(kc, vc, table, lens):
    """NaN keys and values in every row that no query sees (behind lens[n])."""
    page = kc.shape[1]
    for n, L in enumerate(lens):
        cols = 1 if table is None else table.shape[1]
        for s in range(L, cols * page):
            p = n if table is None else int(table[n, s // page])
            kc[p, s % page] = math.nan
            vc[p, s % page] = math.inf


# nseq, nq, L, page, Hq, heads, d, dtype, layout, mask, cap, bias
CASES = {
    "one_key": (1, 1, 1, 1, 1, 1, 64, BF, "token", "causal", 0.0, False),
    "decode_mha": (3, 1, 200, 16, 4, 4, 64, FP, "token", "causal", 0.0, False),
    "decode_gqa8": (5, 1, 700, 64, 16, 2, 128, BF, "token", "causal", 0.0, False),
    "decode_group7": (2, 1, 333, 48, 21, 3, 128, FP, "head", "causal", 30.0, False),
    "decode_group24": (2, 1, 515, 33, 24, 1, 64, BF, "head", "causal", 0.0, True),
    "decode_group32_256": (3, 1, 300, 24, 32, 1, 256, BF, "token", "causal", 0.0, False),
    "decode_group40": (2, 1, 290, 16, 80, 2, 128, FP, "token", "causal", 0.0, False),
    "decode_group64": (2, 1, 1000, 64, 64, 1, 128, BF, "token", "causal", 20.0, True),
    "decode_group64_256": (1, 1, 400, 64, 64, 1, 256, FP, "token", "causal", 0.0, False),
    "decode_group100": (1, 1, 300, 7, 100, 1, 64, BF, "token", "causal", 0.0, False),
    "decode_group130": (2, 1, 200, 16, 130, 1, 128, BF, "token", "causal", 0.0, False),
    "decode_group300_256": (1, 1, 77, 16, 300, 1, 256, FP, "token", "causal", 10.0, False),
    "step_of_5": (3, 5, 260, 32, 6, 2, 128, FP, "token", "causal", 0.0, False),
    "step_of_3_256": (2, 3, 150, 16, 8, 1, 256, BF, "head", "prefix", 0.0, True),
    "prompt": (1, 300, 300, 64, 4, 1, 128, BF, "token", "causal", 0.0, False),
    "prompt_cap": (2, 150, 180, 24, 6, 2, 64, FP, "head", "causal", 50.0, False),
    "prompt_docs": (2, 257, 257, 48, 4, 2, 128, FP, "token", "documents", 0.0, True),
    "prompt_prefix_256": (1, 130, 140, 64, 2, 2, 256, BF, "token", "prefix", 0.0, False),
    "prompt_window_group3": (1, 700, 700, 64, 3, 1, 64, BF, "token", "window", 0.0, False),
    "prompt_direct_mqa": (1, 520, 520, 128, 12, 1, 128, BF, "token", "causal", 0.0, True),
    "decode_direct": (530, 1, 40, 16, 2, 1, 64, FP, "token", "causal", 0.0, False),
    "direct_256": (130, 4, 30, 8, 4, 2, 256, BF, "head", "documents", 15.0, False),
    "rows_no_table": (3, 2, 210, 0, 8, 2, 128, BF, "token", "causal", 0.0, False),
}


def build(case, seed=0):
    nseq, nq, L, page, Hq, heads, d, dtype, layout, mask, cap, bias = case
    g = torch.Generator().manual_seed(seed)
    paged = page > 0
    page = page or L
    cols = -(-L // page)
    kc, vc, table = cache(g, nseq, cols, page, heads, d, dtype, layout, paged=paged)
    lens = [max(nq, L - (n * 37) % max(1, L // 2)) for n in range(nseq)]
    seq, start, length, pos = [], [], [], []
    for n in range(nseq):
        for i in range(nq):
            p = lens[n] - nq + i
            a, b = 0, p + 1
            if mask == "documents":
                a = p // 50 * 50
                if p % 11 == 5:
                    a = b + 3                       # a row that sees nothing
            elif mask == "prefix":
                b = min(lens[n], max(b, lens[n] // 2))
            elif mask == "window":
                a = max(0, p - 20)
            seq.append(n)
            start.append(a)
            length.append(b)
            pos.append(p)
    q = (torch.randn(nseq * nq, Hq, d, generator=g) * 1.5).to(dtype).cuda()
    if nseq < 20:
        poison_behind(kc, vc, table, [max([length[i] for i in range(len(seq)) if seq[i] == n]) for n in range(nseq)])
    kw = dict(table=table, q_start=ints(start) if mask in ("documents", "window") else None, cap=cap,
              slopes=(2.0 ** (-8.0 * torch.arange(1, Hq + 1) / Hq)).float().cuda() if bias else None,
              q_pos=ints(pos) if bias else None)
    return q, kc, vc, ints(seq), ints(length), kw


@pytest.mark.parametrize("name", list(CASES))
def test_attend(name):
    print(f"[attend] {name} {CASES[name]}", flush=True)
    q, kc, vc, seq, length, kw = build(CASES[name])
    got = M.attend(q, kc, vc, seq, length, want_lse=True, **kw)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, seq, length, **kw), name)


def test_empty_batch_and_empty_rows():
    g = torch.Generator().manual_seed(1)
    kc, vc, table = cache(g, 3, 4, 16, 2, 64, BF)
    q = torch.randn(6, 4, 64, generator=g).to(BF).cuda()
    out, lse = M.attend(q[:0], kc, vc, ints([]), ints([]), table=table, want_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    # length zero, a sequence out of range (both sides), a negative length, one beyond the table, a start behind the end
    seq, length = ints([0, -1, 3, 1, 2, 0]), ints([0, 5, 5, -4, 1000, 7])
    start = ints([0, 0, 0, 0, 60, 9])
    got = M.attend(q, kc, vc, seq, length, table=table, q_start=start, want_lse=True)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, seq, length, table=table, q_start=start), "empty rows")
    assert bool((got[0][[0, 1, 2, 3, 5]] == 0).all()) and bool((got[1][[0, 1, 2, 3, 5]] == -math.inf).all())


def test_pages_that_are_none():
    """Table entries outside the pool hide their tokens, whatever the other pages hold."""
    g = torch.Generator().manual_seed(2)
    kc, vc, table = cache(g, 2, 12, 16, 2, 128, FP)
    table[0, 3], table[0, 11], table[1, 0], table[1, 5:] = -1, kc.shape[0], 1 << 30, -7
    q = torch.randn(2, 8, 128, generator=g).to(FP).cuda()
    seq, length = ints([0, 1]), ints([190, 150])
    got = M.attend(q, kc, vc, seq, length, table=table, want_lse=True)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, seq, length, table=table), "no page")


def test_queries_in_any_order():
    """Sequences that alternate within a row tile, one of them out of range."""
    g = torch.Generator().manual_seed(3)
    kc, vc, table = cache(g, 3, 8, 32, 1, 128, BF)
    T = 70
    seq = ints([(0, 0, 1, -1, 2, 2, 2)[t % 7] for t in range(T)])
    length = ints([(t * 29) % 256 for t in range(T)])
    q = torch.randn(T, 4, 128, generator=g).to(BF).cuda()
    got = M.attend(q, kc, vc, seq, length, table=table, want_lse=True)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, seq, length, table=table), "any order")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nq", [1, 5, 12, 25, 60, 300])
def test_large_scores_and_nan_of_visible_values(nq, d):
    """Scores of +-hundreds (weights that vanish) stay finite; a NaN value reaches
    exactly the queries that see it, an infinite one gives an infinity."""
    g = torch.Generator().manual_seed(4)
    L = 200 + nq
    kc, vc, table = cache(g, 1, -(-L // 32), 32, 1, d, BF)
    q = (torch.randn(nq, 2, d, generator=g) * 30).to(BF).cuda()
    length = ints([L - nq + i + 1 for i in range(nq)])
    seq = ints([0] * nq)
    got = M.attend(q, kc, vc, seq, length, table=table, want_lse=True)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, seq, length, table=table), "large scores")
    bad = L - nq // 2 - 1                                         # the first half does not see it
    q2 = (q.float() / 30).to(BF)
    want = A.attend(q2, kc, vc, seq, length, table=table)
    vc[int(table[0, bad // 32]), bad % 32, 0, 5] = math.nan
    vc[int(table[0, bad // 32]), bad % 32, 0, 9] = math.inf
    vc[int(table[0, bad // 32]), bad % 32, 0, 11] = -math.inf
    out, lse = M.attend(q2, kc, vc, seq, length, table=table, want_lse=True)
    torch.cuda.synchronize()
    sees = (length > bad).cpu()
    o = out.cpu().float()
    assert bool(torch.isnan(o[sees][..., 5]).all())
    assert bool((o[sees][..., 9] == math.inf).all()) and bool((o[sees][..., 11] == -math.inf).all())
    for i in (5, 9, 11):                # everything else as without them
        out[sees.cuda(), :, i] = want[0][sees][..., i].to(BF).cuda()
    A.check((out, lse), want, "around a NaN")


@pytest.mark.parametrize("name", ["prompt_docs", "prompt_window_group3", "prompt_prefix_256", "direct_256"])
def test_values_outside_the_interval_may_be_anything(name):
    """NaN and infinities in the values of tokens that some queries of a row tile
    see and others do not (other documents, tokens behind the window)."""
    q, kc, vc, seq, length, kw = build(CASES[name])
    start = kw["q_start"] if kw["q_start"] is not None else torch.zeros_like(length)
    clean = A.attend(q, kc, vc, seq, length, **kw)
    page, table = kc.shape[1], kw["table"]
    bad = [100, 117, 121] if name == "prompt_prefix_256" else [3, 57, 120]   # behind the prefix that all see
    for n in range(min(3, table.shape[0])):
        for s in bad:
            if s // page < table.shape[1]:
                vc[int(table[n, s // page]), s % page] = math.nan if s % 2 else math.inf
    out, lse = M.attend(q, kc, vc, seq, length, want_lse=True, **kw)
    torch.cuda.synchronize()
    sees = torch.zeros(len(length), dtype=torch.bool)
    for s in bad:
        sees |= ((start <= s) & (s < length) & (seq < 3)).cpu()
    assert bool((~sees).any())
    A.check((out[~sees.cuda()], lse[~sees.cuda()]), tuple(x[~sees] for x in clean), name)
    assert not bool(torch.isfinite(out[sees.cuda()].float()).all()) or not bool(sees.any())


@pytest.mark.parametrize("Hq,d", [(8, 128), (64, 128), (64, 64), (40, 256), (100, 128)])
def test_windows_of_single_queries(Hq, d):
    """A decode step with sliding windows: what lies before a window may hold anything."""
    g = torch.Generator().manual_seed(31)
    kc, vc, table = cache(g, 4, 10, 32, 1, d, BF)
    q = torch.randn(4, Hq, d, generator=g).to(BF).cuda()
    seq, length, start = ints([0, 1, 2, 3]), ints([300, 77, 130, 320]), ints([171, 76, 100, 319])
    want = A.attend(q, kc, vc, seq, length, table=table, q_start=start)
    for n in range(4):
        for s in range(max(0, int(start[n]) - 40), int(start[n])):
            kc[int(table[n, s // 32]), s % 32] = math.nan
            vc[int(table[n, s // 32]), s % 32] = math.nan if s % 2 else -math.inf
    got = M.attend(q, kc, vc, seq, length, table=table, q_start=start, want_lse=True)
    torch.cuda.synchronize()
    A.check(got, want, "windows")


@pytest.mark.parametrize("cap", [0.5, 3.0, 40.0, 300.0, 20000.0])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("nq", [1, 40])
def test_caps(cap, bias, nq):
    """Caps that most scores pass, caps that none comes near, and large ones."""
    g = torch.Generator().manual_seed(41)
    kc, vc, table = cache(g, 2, 20, 16, 2, 128, FP)
    q = (torch.randn(2 * nq, 8, 128, generator=g) * 4).to(FP).cuda()
    q[0] *= 0.01                                            # scores near zero
    seq = ints([0] * nq + [1] * nq)
    length = ints([320 - nq + i + 1 for i in range(nq)] * 2)
    kw = dict(table=table, cap=cap, slopes=torch.linspace(0.0, 0.3, 8).cuda() if bias else None)
    got = M.attend(q, kc, vc, seq, length, want_lse=True, **kw)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, seq, length, **kw), f"cap {cap}")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [20, 64])
@pytest.mark.parametrize("nq", [3, 320])
def test_caps_by_size_of_the_scores(nq, page, d):
    """Row tiles of small, middling and large scores against one cap: up to 0.18, up to
    0.35 and beyond of it, which take different forms; pages that hold whole groups of
    rows and others."""
    g = torch.Generator().manual_seed(43)
    kc, vc, table = cache(g, 1, (400 + page - 1) // page, page, 2, d, BF)
    q = torch.randn(nq, 16, d, generator=g)
    sizes = [0.05, 1.0, 1.8, 8.0]
    for i in range(nq):
        q[i] *= sizes[i * 4 // nq]
    q = q.to(BF).cuda()
    seq, length = ints([0] * nq), ints([400 - nq + i + 1 for i in range(nq)])
    kw = dict(table=table, cap=24.0)
    got = M.attend(q, kc, vc, seq, length, want_lse=True, **kw)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, seq, length, **kw), f"d {d} page {page}")


def test_infinite_scores_of_visible_keys():
    """Keys that overflow to infinity: NaN as in the formula without a cap, the cap
    itself with one; rows of other heads and queries stay."""
    g = torch.Generator().manual_seed(42)
    kc, vc, table = cache(g, 1, 4, 16, 2, 64, BF)
    q = torch.randn(3, 4, 64, generator=g).to(BF).cuda()
    seq, length = ints([0, 0, 0]), ints([20, 30, 40])
    clean = A.attend(q, kc, vc, seq, length, table=table)
    kc[int(table[0, 1]), 9, 0] = math.inf                   # token 25 of the first kv head
    q[:, :2] = q[:, :2].abs() + 0.1
    want = A.attend(q[:, 2:], kc[:, :, 1:], vc[:, :, 1:], seq, length, table=table)
    out, lse = M.attend(q, kc, vc, seq, length, table=table, want_lse=True)
    capped, _ = M.attend(q, kc, vc, seq, length, table=table, cap=10.0)
    torch.cuda.synchronize()
    assert bool(torch.isnan(out[1:, :2]).all()) and bool(torch.isfinite(out[0]).all())
    A.check((out[:, 2:], lse[:, 2:]), want, "other heads")
    assert bool(torch.isfinite(capped).all())


def test_stream_argument():
    """A call on a stream of the caller's, its workspace made by the call, while the
    current stream goes on allocating."""
    q, kc, vc, seq, length, kw = build(CASES["decode_gqa8"])
    want = M.attend(q, kc, vc, seq, length, want_lse=True, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        got = M.attend(q, kc, vc, seq, length, want_lse=True, stream=side, **kw)
        junk = [torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        del junk


def test_same_call_twice_and_dirty_workspace():
    """The same bits again, whatever the workspace held before, and without lse."""
    q, kc, vc, seq, length, kw = build(CASES["decode_gqa8"])
    need = M.attend_workspace_bytes(M.OP_ATTEND, q.shape[0], q.shape[1], 2, 128, 5)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    a = M.attend(q, kc, vc, seq, length, want_lse=True, ws=ws, **kw)
    b = M.attend(q, kc, vc, seq, length, want_lse=True, ws=ws, **kw)
    c, none = M.attend(q, kc, vc, seq, length, **kw)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[0], c) and none is None


def test_query_slices_and_given_outputs():
    """Queries as a slice of a fused projection, outputs into rows of a larger buffer."""
    q, kc, vc, seq, length, kw = build(CASES["step_of_5"])
    T, Hq, d = q.shape
    fused = torch.full((T, Hq + 5, d), math.nan, dtype=q.dtype, device="cuda")
    fused[:, 2:2 + Hq] = q
    big = torch.full((T + 3, Hq, d), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((T + 3, Hq), 7.0, device="cuda")
    out, l = M.attend(fused[:, 2:2 + Hq], kc, vc, seq, length, out=big[:T], lse=lse[:T], **kw)
    torch.cuda.synchronize()
    A.check((out, l), A.attend(q, kc, vc, seq, length, **kw), "slices")
    assert bool((big[T:] == 7).all()) and bool((lse[T:] == 7).all())


def test_graph_replays_and_streams():
    """Captured once and replayed over new lengths and queries, against eager calls on another stream."""
    q, kc, vc, seq, length, kw = build(CASES["decode_mha"])
    for x in (kc, vc):
        x.copy_(torch.randn_like(x, dtype=torch.float32))
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ws = torch.empty(M.attend_workspace_bytes(M.OP_ATTEND, q.shape[0], q.shape[1], 4, 64, 3), dtype=torch.uint8, device="cuda")
    M.attend(q, kc, vc, seq, length, out=out, lse=lse, ws=ws, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.attend(q, kc, vc, seq, length, out=out, lse=lse, ws=ws, **kw)
    side = torch.cuda.Stream()
    for i in range(4):
        q.copy_(torch.randn_like(q, dtype=torch.float32))
        length.copy_(ints([200 - 60 * i, 1 + i, 7 * i]))
        graph.replay()
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            o2, l2 = M.attend(q, kc, vc, seq, length, want_lse=True, **kw)
        side.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        A.check((out, lse), A.attend(q, kc, vc, seq, length, **kw), f"replay {i}")


@pytest.mark.parametrize("nq", [1, 40])
def test_rows_behind_32_bits(nq):
    """Keys and values beyond 2^32 elements of their caches, for small and large row tiles."""
    npages = 66000
    g = torch.Generator().manual_seed(9)
    kc = torch.empty(npages, 64, 8, 128, dtype=BF, device="cuda")
    vc = torch.empty(npages, 64, 8, 128, dtype=BF, device="cuda")
    assert kc.numel() > 2 ** 32
    used = torch.tensor([npages - 1, 0, 32768, npages - 2])
    for x in (kc, vc):
        x[used.cuda()] = torch.randn(4, 64, 8, 128, generator=g).to(BF).cuda()
    q = torch.randn(nq, 64, 128, generator=g).to(BF).cuda()
    small = ints([[0, 1, 2, 3]])
    args = ints([0] * nq), ints([250 - nq + i + 1 for i in range(nq)])
    got = M.attend(q, kc, vc, *args, table=used[None].to(torch.int32).cuda(), want_lse=True)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc[used.cuda()], vc[used.cuda()], *args, table=small), "behind 32 bits")


# ---------------------------------------------------------------- selected tokens
SELECTED = {
    # T, nseq, L, page, topk, Hq, heads, d, dtype, cap, bias
    "one": (1, 1, 5, 2, 1, 1, 1, 64, BF, 0.0, False),
    "mqa64": (3, 3, 900, 64, 300, 64, 1, 128, BF, 0.0, False),
    "gqa8": (10, 2, 500, 16, 129, 16, 2, 128, FP, 25.0, True),
    "group20_256": (4, 2, 300, 48, 64, 20, 1, 256, BF, 0.0, True),
    "group200": (2, 1, 300, 16, 65, 200, 1, 64, FP, 0.0, False),
    "direct": (600, 2, 128, 16, 33, 4, 1, 64, BF, 0.0, False),
}


@pytest.mark.parametrize("name", list(SELECTED))
def test_attend_selected(name):
    T, nseq, L, page, topk, Hq, heads, d, dtype, cap, bias = SELECTED[name]
    print(f"[selected] {name} {SELECTED[name]}", flush=True)
    g = torch.Generator().manual_seed(11)
    kc, vc, table = cache(g, nseq, -(-L // page), page, heads, d, dtype)
    seq = torch.arange(T) % nseq
    length = torch.tensor([max(1, L - 17 * t % L) for t in range(T)])
    # any order, repeats, padding and ids out of range between them
    idx = torch.randint(-2, L + 5, (T, topk), generator=g).to(torch.int32)
    idx[:, topk - topk // 4:] = -1
    if topk > 3:
        idx[0, 1] = idx[0, 0] = 0
        idx[-1, :] = -1                     # a query with nothing selected
    q = torch.randn(T, Hq, d, generator=g).to(dtype).cuda()
    slopes = torch.linspace(0.01, 0.2, Hq).cuda() if bias else None
    kw = dict(table=table, cap=cap, slopes=slopes)
    got = M.attend_selected(q, kc, vc, idx.cuda(), ints(seq), ints(length), want_lse=True, **kw)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, seq, length, idx=idx, **kw), name)


def test_selecting_everything_is_attending_to_it():
    q, kc, vc, seq, length, kw = build(CASES["decode_gqa8"])
    idx = torch.arange(700, dtype=torch.int32, device="cuda").expand(5, 700).contiguous()
    a = M.attend(q, kc, vc, seq, length, want_lse=True, **kw)
    kw.pop("q_start"), kw.pop("q_pos")
    b = M.attend_selected(q, kc, vc, idx, seq, length, want_lse=True, **kw)
    torch.cuda.synchronize()
    A.check(b, A.attend(q, kc, vc, seq, length, **kw), "everything")
    A.check(a, A.attend(q, kc, vc, seq, length, **kw), "attend")


# ---------------------------------------------------------------- shared prefixes
SHARED = {
    # npre, nseq, nq, P, L, page, Hq, heads, d, dtype, cap, bias
    "one_of_each": (1, 1, 1, 1, 1, 1, 1, 1, 64, BF, 0.0, False),
    "samples": (1, 12, 1, 700, 90, 16, 8, 2, 128, BF, 0.0, False),
    "two_prompts": (2, 6, 1, 333, 50, 24, 21, 3, 64, FP, 30.0, True),
    "steps": (3, 6, 3, 200, 40, 8, 8, 1, 256, BF, 0.0, True),
    "mqa": (2, 5, 1, 300, 33, 64, 64, 1, 128, FP, 0.0, False),
    "direct": (2, 140, 4, 130, 20, 16, 4, 2, 64, BF, 0.0, False),
}


@pytest.mark.parametrize("name", list(SHARED))
def test_attend_shared(name):
    npre, nseq, nq, P, L, page, Hq, heads, d, dtype, cap, bias = SHARED[name]
    print(f"[shared] {name} {SHARED[name]}", flush=True)
    g = torch.Generator().manual_seed(21)
    pc, oc = -(-P // page), -(-L // page)
    npages = npre * pc + nseq * oc + 2
    order = torch.randperm(npages, generator=g).to(torch.int32)
    pre_table, table = order[:npre * pc].view(npre, pc).cuda(), order[npre * pc:npre * pc + nseq * oc].view(nseq, oc).cuda()
    kc, vc = (torch.randn(npages, page, heads, d, generator=g).to(dtype).cuda() for _ in range(2))
    T = nseq * nq
    seq = torch.arange(nseq).repeat_interleave(nq)
    pre = (torch.arange(nseq) * npre // nseq).repeat_interleave(nq)
    length = torch.tensor([max(0, L - (7 * n) % (L + 1)) for n in range(nseq)]).repeat_interleave(nq)
    pre_len = torch.tensor([max(0, P - 100 * i) for i in range(npre)])
    if T > 3:
        pre[1], pre[2] = -1, npre               # no prefix
        seq[3] = -1                             # a padding row
        length[1] = 0                           # nothing at all
    q = torch.randn(T, Hq, d, generator=g).to(dtype).cuda()
    slopes = torch.linspace(0.01, 0.2, Hq).cuda() if bias else None
    kw = dict(table=table, pre_table=pre_table, cap=cap, slopes=slopes)
    got = M.attend_shared(q, kc, vc, ints(seq), ints(length), ints(pre), ints(pre_len), want_lse=True, **kw)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, seq, length, pre=pre, pre_len=pre_len, **kw), name)


def test_shared_without_tables():
    """Prefixes and sequences as rows of one cache."""
    g = torch.Generator().manual_seed(22)
    kc, vc = (torch.randn(6, 150, 2, 64, generator=g).to(BF).cuda() for _ in range(2))
    q = torch.randn(4, 4, 64, generator=g).to(BF).cuda()
    args = (ints([2, 3, 4, 5]), ints([10, 150, 0, 77]), ints([0, 0, 1, 1]), ints([150, 64]))
    got = M.attend_shared(q, kc, vc, *args, want_lse=True)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, args[0], args[1], pre=args[2], pre_len=args[3]), "rows")
