"""Forms of the kernels by cap, bias, tile and layout, each over whole runs of keys
and their ends: capped scores in tiles of 64 rows, of selected tokens and behind
prefixes; every one of small, middling and large scores against the cap."""
import pytest
import torch

import attend_oracle as A
from routed_token_indexer_amd import _lib as M

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
SIZES = [0.05, 1.0, 1.8, 8.0]     # of the queries: scores up to 0.18, 0.35 and beyond of a cap of 24


def ints(v):
    return torch.as_tensor(v, dtype=torch.int32).cuda()


def paged(g, pages, page, heads, d, dtype, layout="token"):
    kv = []
    for _ in range(2):
        x = torch.randn(pages, page, heads, d, generator=g).to(dtype).cuda()
        kv.append(x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) if layout == "head" else x)
    return kv


def queries(g, n, Hq, d, dtype, size):
    q = torch.randn(n, Hq, d, generator=g)
    for i in range(n):
        q[i] *= SIZES[i * 4 // n] if size is None else size
    return q.to(dtype).cuda()


@pytest.mark.parametrize("size", [None, *SIZES])
@pytest.mark.parametrize("cap", [0.0, 24.0, 300.0])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("page", [20, 64])
@pytest.mark.parametrize("d,dtype", [(64, FP), (128, BF), (128, FP), (256, BF)])
def test_tiles_of_64_rows(d, dtype, page, bias, cap, size):
    nq, Hq, heads, L = 7, 16, 2, 500
    g = torch.Generator().manual_seed(101)
    cols = -(-L // page)
    kc, vc = paged(g, 2 * cols, page, heads, d, dtype, "head" if page == 20 else "token")
    table = torch.randperm(2 * cols, generator=g).view(2, cols).to(torch.int32).cuda()
    q = queries(g, 2 * nq, Hq, d, dtype, size)
    seq = ints([0] * nq + [1] * nq)
    length = ints([L - nq + i + 1 for i in range(nq)] + [301 + i for i in range(nq)])
    kw = dict(table=table, cap=cap, slopes=torch.linspace(0.0, 0.05, Hq).cuda() if bias else None)
    got = M.attend(q, kc, vc, seq, length, want_lse=True, **kw)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, seq, length, **kw), "64 rows")


@pytest.mark.parametrize("size", [None, *SIZES])
@pytest.mark.parametrize("cap", [24.0, 300.0])
@pytest.mark.parametrize("T", [5, 270])
@pytest.mark.parametrize("Hq,heads,d,dtype", [(8, 2, 64, BF), (24, 1, 128, FP), (64, 1, 128, BF), (30, 1, 256, BF), (100, 1, 64, FP)])
def test_selected(Hq, heads, d, dtype, T, cap, size):
    L, page, topk = 400, 16, 150
    g = torch.Generator().manual_seed(102)
    cols = L // page
    kc, vc = paged(g, 2 * cols, page, heads, d, dtype)
    table = torch.randperm(2 * cols, generator=g).view(2, cols).to(torch.int32).cuda()
    q = queries(g, T, Hq, d, dtype, size)
    idx = torch.stack([torch.randperm(L, generator=g)[:topk] for _ in range(T)]).to(torch.int32)
    idx[0, 130:] = -1
    seq, length = ints([t % 2 for t in range(T)]), ints([L if t % 3 else 200 for t in range(T)])
    kw = dict(table=table, cap=cap)
    got = M.attend_selected(q, kc, vc, idx.cuda(), seq, length, want_lse=True, **kw)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, seq, length, idx=idx, **kw), "selected")


@pytest.mark.parametrize("size", [None, *SIZES])
@pytest.mark.parametrize("cap", [24.0, 300.0])
@pytest.mark.parametrize("nseq,nq", [(3, 1), (9, 2), (90, 3)])
@pytest.mark.parametrize("Hq,heads,d,dtype,page", [(8, 2, 64, BF, 16), (16, 2, 128, FP, 64), (16, 1, 256, BF, 20)])
def test_shared(Hq, heads, d, dtype, page, nseq, nq, cap, size):
    P, L = 300, 70
    g = torch.Generator().manual_seed(103)
    pc, oc = -(-P // page), -(-L // page)
    kc, vc = paged(g, 2 * pc + nseq * oc, page, heads, d, dtype)
    order = torch.randperm(2 * pc + nseq * oc, generator=g).to(torch.int32)
    pre_table, table = order[:2 * pc].view(2, pc).cuda(), order[2 * pc:].view(nseq, oc).cuda()
    T = nseq * nq
    q = queries(g, T, Hq, d, dtype, size)
    seq = torch.arange(nseq).repeat_interleave(nq)
    args = (ints(seq), ints([max(0, L - (7 * t) % (L + 1)) for t in range(T)]), ints(seq * 2 // nseq), ints([P, 133]))
    kw = dict(table=table, pre_table=pre_table, cap=cap)
    got = M.attend_shared(q, kc, vc, *args, want_lse=True, **kw)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, args[0], args[1], pre=args[2], pre_len=args[3], **kw), "shared")
