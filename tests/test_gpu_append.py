"""misa_cache_append against the plain rotation in fp64: both pairings, partial
rotation, page sizes, layouts and strides, skipped tokens, untouched rows."""
import pytest
import torch

import attend_oracle as A
from routed_token_indexer_amd import _lib as M

pytestmark = pytest.mark.gpu


def table_of(P, rot, dev="cuda"):
    h = rot // 2
    ang = torch.arange(P, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(h, dtype=torch.float64) / h)
    return torch.cat([ang.cos(), ang.sin()], 1).float().to(dev)


def make(nseq, cols, page, heads, d, dtype, layout, seed=0, values=True):
    g = torch.Generator().manual_seed(seed)
    npages = nseq * cols + 3
    shape = (npages, heads, page, d) if layout == "head" else (npages, page, heads, d)
    kv = [torch.randn(shape, generator=g).to(dtype).cuda() for _ in range(2 if values else 1)]
    if layout == "head":
        kv = [x.permute(0, 2, 1, 3) for x in kv]
    table = torch.randperm(npages, generator=g)[:nseq * cols].view(nseq, cols).to(torch.int32).cuda()
    return kv[0], kv[1] if values else None, table


CASES = [
    # nseq, nq, page, heads, Hq, d, rot, interleaved, dtype, layout
    (1, 1, 1, 1, 1, 64, 64, False, torch.bfloat16, "token"),
    (64, 1, 64, 8, 64, 128, 128, False, torch.bfloat16, "token"),
    (3, 50, 16, 2, 6, 128, 64, True, torch.float16, "head"),
    (2, 129, 48, 5, 35, 256, 16, False, torch.float16, "token"),
    (4, 7, 24, 1, 7, 32, 32, True, torch.bfloat16, "head"),
    (1, 300, 128, 3, 0, 64, 32, False, torch.bfloat16, "token"),
    (2, 9, 5, 1, 128, 1024, 1024, True, torch.float16, "token"),
    (5, 3, 7, 2, 4, 48, 16, False, torch.bfloat16, "head"),
    (1, 1000, 64, 8, 8, 128, 0, False, torch.bfloat16, "token"),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_append(case):
    nseq, nq, page, heads, Hq, d, rot, inter, dtype, layout = case
    print(f"[append] {case}", flush=True)
    cols = -(-(nq + 2 * page) // page)
    kc, vc, table = make(nseq, cols, page, heads, d, dtype, layout)
    g = torch.Generator().manual_seed(7)
    N = nseq * nq
    fused = torch.randn(N, Hq + 2 * heads, d, generator=g).to(dtype).cuda()     # one projection, sliced
    q, k, v = fused[:, :Hq] if Hq else None, fused[:, Hq:Hq + heads], fused[:, Hq + heads:]
    tok = torch.cat([torch.arange(nq) + (n * 13) % (cols * page - nq + 1) for n in range(nseq)]).to(torch.int32)
    seq = torch.arange(nseq, dtype=torch.int32).repeat_interleave(nq)
    perm = torch.randperm(N, generator=g)                                       # tokens in any order
    tok, seq = tok[perm], seq[perm]
    cs = table_of(cols * page, rot) if rot else None
    want_k, want_v = kc.cpu().double(), vc.cpu().double()
    tol_k = torch.zeros_like(want_k)
    at = (table.cpu()[seq.long(), tok.long() // page].long(), tok.long() % page)
    if rot:
        yk, tk = A.rotate(k.cpu(), cs.cpu(), tok.long(), inter)
    else:
        yk, tk = k.cpu().double(), torch.zeros(k.shape, dtype=torch.float64)
    want_k[at], tol_k[at] = yk, tk
    want_v[at] = v.cpu().double()
    out = M.cache_append(k, v, kc, vc, seq.cuda(), tok.cuda(), table=table, q=q, cos_sin=cs, interleaved=inter)
    torch.cuda.synchronize()
    assert bool(((kc.cpu().double() - want_k).abs() <= tol_k).all())            # other rows: exactly as they were
    assert torch.equal(vc.cpu().double(), want_v)
    if Hq:
        yq, tq = A.rotate(q.cpu(), cs.cpu(), tok.long(), inter) if rot else (q.cpu().double(), torch.zeros(q.shape))
        assert bool(((out.cpu().double() - yq).abs() <= tq).all())
    else:
        assert out is None


def test_skipped_tokens_leave_everything():
    """Bad sequence, index, page or position: the cache and the query row keep their values."""
    kc, vc, table = make(3, 4, 16, 2, 64, torch.bfloat16, "token")
    table[1, 2] = -1
    table[2, 0] = kc.shape[0]
    seq = torch.tensor([0, -1, 3, 0, 0, 1, 2, 1, 0], dtype=torch.int32)
    tok = torch.tensor([5, 5, 5, -1, 64, 40, 3, 20, 50], dtype=torch.int32)
    good = torch.tensor([1, 0, 0, 0, 0, 0, 0, 1, 0], dtype=torch.bool)            # the last one: position 50 >= P
    cs = table_of(40, 64)
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(9, h, 64, generator=g).to(torch.bfloat16).cuda() for h in (4, 2, 2))
    q_out = torch.full_like(q, 7.0)
    want_k, want_v, want_q = kc.cpu().double(), vc.cpu().double(), q_out.cpu().double()
    tol_k, tol_q = torch.zeros_like(want_k), torch.zeros_like(want_q)
    yk, tk = A.rotate(k.cpu(), cs.cpu(), tok.long().clamp(0, 39), False)
    yq, tq = A.rotate(q.cpu(), cs.cpu(), tok.long().clamp(0, 39), False)
    for i in range(9):
        if good[i]:
            p, s = int(table[seq[i], tok[i] // 16]), int(tok[i] % 16)
            want_k[p, s], tol_k[p, s], want_v[p, s] = yk[i], tk[i], v[i].cpu().double()
            want_q[i], tol_q[i] = yq[i], tq[i]
    M.cache_append(k, v, kc, vc, seq.cuda(), tok.cuda(), table=table, q=q, q_out=q_out, cos_sin=cs)
    torch.cuda.synchronize()
    assert bool(((kc.cpu().double() - want_k).abs() <= tol_k).all())
    assert torch.equal(vc.cpu().double(), want_v)
    assert bool(((q_out.cpu().double() - want_q).abs() <= tol_q).all())


def test_positions_apart_from_indices_and_in_place_queries():
    """Rotary positions of their own, queries turned in place, keys alone in the
    indexer's layout k [nseq, Lmax, d]."""
    k_cache = torch.zeros(3, 100, 128, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(5)
    k = torch.randn(6, 1, 128, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(6, 8, 128, generator=g).to(torch.bfloat16).cuda()
    seq = torch.tensor([0, 0, 1, 1, 2, 2], dtype=torch.int32).cuda()
    tok = torch.tensor([0, 1, 50, 51, 98, 99], dtype=torch.int32).cuda()
    pos = torch.tensor([4000, 0, 1, 3999, 17, 18], dtype=torch.int32).cuda()
    cs = table_of(4001, 64)
    q0 = q.clone()
    yk, tk = A.rotate(k.cpu(), cs.cpu(), pos.cpu().long(), True)
    yq, tq = A.rotate(q0.cpu(), cs.cpu(), pos.cpu().long(), True)
    out = M.cache_append(k, None, k_cache, None, seq, tok, q=q, q_out=q, cos_sin=cs, pos=pos, interleaved=True)
    torch.cuda.synchronize()
    assert out is q
    got = k_cache.cpu().double()
    assert bool(((got[seq.cpu().long(), tok.cpu().long()] - yk[:, 0]).abs() <= tk[:, 0]).all())
    assert int((got.abs().sum(-1) > 0).sum()) == 6
    assert bool(((q.cpu().double() - yq).abs() <= tq).all())


def test_rows_behind_32_bits():
    """A cache whose last pages lie beyond 2^32 elements."""
    npages = 66000
    kc = torch.empty(npages, 64, 8, 128, dtype=torch.bfloat16, device="cuda")
    assert kc.numel() > 2 ** 32
    table = torch.tensor([[npages - 1, 0], [npages - 2, 32769]], dtype=torch.int32, device="cuda")
    kc[table.flatten().long()] = 0
    k = torch.randn(4, 8, 128, device="cuda").to(torch.bfloat16)
    seq = torch.tensor([0, 0, 1, 1], dtype=torch.int32, device="cuda")
    tok = torch.tensor([63, 64, 0, 127], dtype=torch.int32, device="cuda")
    M.cache_append(k, None, kc, None, seq, tok, table=table)
    torch.cuda.synchronize()
    for i, (p, s) in enumerate([(npages - 1, 63), (0, 0), (npages - 2, 0), (32769, 63)]):
        assert torch.equal(kc[p, s], k[i])
    assert int((kc[table.flatten().long()].abs().sum((2, 3)) > 0).sum()) == 4


def test_graph_and_streams():
    """Captured once, replayed with new inputs in the same tensors, and launched on a stream of the caller's."""
    kc, vc, table = make(4, 3, 16, 2, 128, torch.bfloat16, "head")
    cs = table_of(48, 128)
    seq = torch.arange(4, dtype=torch.int32, device="cuda")
    tok = torch.zeros(4, dtype=torch.int32, device="cuda")
    k, v = (torch.randn(4, 2, 128, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(4, 16, 128, device="cuda").to(torch.bfloat16)
    q_out = torch.empty_like(q)
    M.cache_append(k, v, kc, vc, seq, tok, table=table, q=q, q_out=q_out, cos_sin=cs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.cache_append(k, v, kc, vc, seq, tok, table=table, q=q, q_out=q_out, cos_sin=cs)
    kc2, vc2 = kc.clone(), vc.clone()
    kc2, vc2 = torch.empty_strided(kc.shape, kc.stride(), dtype=kc.dtype, device="cuda"), torch.empty_strided(
        vc.shape, vc.stride(), dtype=vc.dtype, device="cuda")
    kc2.copy_(kc)
    vc2.copy_(vc)
    side = torch.cuda.Stream()
    for i in range(1, 5):
        for x in (k, v, q):
            x.copy_(torch.randn_like(x, dtype=torch.float32))
        tok.fill_(11 * i)
        graph.replay()
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        other = M.cache_append(k, v, kc2, vc2, seq, tok, table=table, q=q, cos_sin=cs, stream=side)
        side.synchronize()
        assert torch.equal(other, q_out) and torch.equal(kc, kc2) and torch.equal(vc, vc2)
