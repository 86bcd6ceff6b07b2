"""Capped scores of rows that see few keys: each score keeps fp32's accuracy of
its own size, with and without a distance bias, and also where a value that the
row does not see is not finite. The log-sum shows it."""
import math

import pytest
import torch

import attend_bounds
import attend_oracle as A
from routed_token_indexer_amd import _lib as M

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def paged(g, nseq, cols, page, heads, d, dtype):
    table = torch.randperm(nseq * cols, generator=g).view(nseq, cols).to(torch.int32).cuda()
    return (*(torch.randn(nseq * cols, page, heads, d, generator=g).to(dtype).cuda() for _ in range(2)), table)


def ints(v):
    return torch.as_tensor(v, dtype=torch.int32).cuda()


# nq, Hq, heads, d, page: tiles of 16, 32, 64 and 128 rows
TILES = [(1, 8, 1, 64, 16), (1, 24, 1, 128, 20), (3, 8, 1, 128, 64), (3, 8, 1, 256, 32), (6, 8, 1, 64, 64), (7, 8, 1, 128, 20),
         (6, 8, 1, 256, 20), (40, 4, 1, 64, 20), (40, 4, 1, 128, 64), (40, 4, 1, 256, 20), (300, 2, 1, 128, 64)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("cap", [4.0, 50.0, 256.0, 1000.0])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("tile", TILES, ids=[f"{t[0]}x{t[1]}-d{t[3]}-p{t[4]}" for t in TILES])
def test_few_keys(monkeypatch, tile, bias, cap, dtype):
    """One to 31 visible keys and scores of hundredths."""
    nq, Hq, heads, d, page = tile
    g = torch.Generator().manual_seed(81)
    kc, vc, table = paged(g, 2, -(-120 // page), page, heads, d, dtype)
    q = (0.03 * torch.randn(2 * nq, Hq, d, generator=g)).to(dtype).cuda()
    seen = [1 + (i * 7) % 31 if i % 5 else 1 for i in range(2 * nq)]
    start = [(i * 13) % 80 for i in range(2 * nq)]
    seq = ints([0] * nq + [1] * nq)
    kw = dict(table=table, q_start=ints(start), cap=cap, slopes=torch.full((Hq,), 1e-5, device="cuda") if bias else None)
    length = ints([a + n for a, n in zip(start, seen)])
    monkeypatch.setattr(A, "one_query", attend_bounds.one_query)
    want = A.attend(q, kc, vc, seq, length, **kw)
    got = M.attend(q, kc, vc, seq, length, want_lse=True, **kw)
    torch.cuda.synchronize()
    A.check(got, want, "few keys")
    # a value that half of the rows do not see: the others' bits may move within the same bound
    v2 = vc.clone()
    for n in range(2):
        s = start[n * nq] + seen[n * nq] - 1
        v2[int(table[n, s // page]), s % page, 0, 0] = math.nan
    got = M.attend(q, kc, v2, seq, length, want_lse=True, **kw)
    torch.cuda.synchronize()
    hit = torch.isnan(got[0]).any(-1).any(-1).cpu()
    s = torch.tensor([start[n * nq] + seen[n * nq] - 1 for n in range(2)])[seq.cpu().long()]
    assert torch.equal(hit, (torch.tensor(start) <= s) & (s < length.cpu()))
    out = torch.where(hit[:, None, None].cuda(), want[0].to(dtype).cuda(), got[0])
    A.check((out, got[1]), want, "beside a NaN")


@pytest.mark.parametrize("cap", [50.0, 256.0])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("Hq,d", [(4, 64), (64, 128), (24, 256)])
def test_few_selected(monkeypatch, Hq, d, bias, cap):
    g = torch.Generator().manual_seed(82)
    kc, vc, table = paged(g, 2, 6, 20, 1, d, BF)
    q = (0.03 * torch.randn(5, Hq, d, generator=g)).to(BF).cuda()
    idx = torch.stack([torch.randperm(100, generator=g)[:29] for _ in range(5)]).to(torch.int32).cuda()
    idx[1, 1:] = -1
    seq, length = ints([0, 1, 1, 0, 1]), ints([100] * 5)
    kw = dict(table=table, cap=cap, slopes=torch.full((Hq,), 1e-5, device="cuda") if bias else None)
    monkeypatch.setattr(A, "one_query", attend_bounds.one_query)
    got = M.attend_selected(q, kc, vc, idx, seq, length, want_lse=True, **kw)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, seq, length, idx=idx, **kw), "few selected")


@pytest.mark.parametrize("cap", [50.0, 256.0])
@pytest.mark.parametrize("bias", [False, True])
def test_few_behind_a_prefix(monkeypatch, bias, cap):
    g = torch.Generator().manual_seed(83)
    kc, vc, table = paged(g, 6, 2, 16, 2, 64, FP)
    q = (0.03 * torch.randn(5, 8, 64, generator=g)).to(FP).cuda()
    args = ints([0, 1, 2, 3, 4]), ints([1, 20, 31, 0, 5]), ints([0, 0, 0, 0, 0]), ints([9])
    kw = dict(table=table[:5].contiguous(), pre_table=table[5:].contiguous(), cap=cap,
              slopes=torch.full((8,), 1e-5, device="cuda") if bias else None)
    monkeypatch.setattr(A, "one_query", attend_bounds.one_query)
    got = M.attend_shared(q, kc, vc, *args, want_lse=True, **kw)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, args[0], args[1], pre=args[2], pre_len=args[3], **kw), "few behind a prefix")
