"""fp16 rows whose result is the sum of very small weights: one key with a value
of zero holds nearly all of the weight, and the others, 12 to 18 below its score,
make the output. The weights' 16 bits must hold them."""
import pytest
import torch

import attend_bounds
import attend_oracle as A
from routed_token_indexer_amd import _lib as M

pytestmark = pytest.mark.gpu
FP = torch.float16

# nq, L, page, Hq, heads, d
SHAPES = {
    "decode": (1, 60, 16, 4, 1, 64),
    "decode_group24": (1, 60, 16, 24, 1, 128),
    "decode_group24_256": (1, 30, 16, 24, 1, 256),
    "step_of_5": (5, 500, 16, 12, 1, 128),
    "prompt": (300, 2500, 64, 2, 1, 64),
    "prompt_128": (270, 1500, 20, 2, 1, 128),
    "prompt_256": (260, 900, 64, 2, 1, 256),
}


def inputs(nq, L, page, Hq, heads, d, above):
    """Scores of about ``above`` for key 0, whose value is zero, and near zero for the others."""
    g = torch.Generator().manual_seed(71)
    cols = -(-L // page)
    table = torch.randperm(cols, generator=g).view(1, cols).to(torch.int32)
    q = 0.3 * torch.randn(nq, Hq, d, generator=g)
    k, v = 0.3 * torch.randn(cols * page, heads, d, generator=g), 1 + 0.25 * torch.randn(cols * page, heads, d, generator=g)
    q[..., 0], k[..., 0] = 4.0, 0.0
    k[0, :, 0], v[0] = above * d ** 0.5 / 4, 0.0
    kc, vc = torch.empty(cols, page, heads, d, dtype=FP), torch.empty(cols, page, heads, d, dtype=FP)
    for x, c in ((k, kc), (v, vc)):
        c[table[0].long()] = x.view(cols, page, heads, d).to(FP)
    return q.to(FP).cuda(), kc.cuda(), vc.cuda(), table.cuda()


@pytest.mark.parametrize("above", [12.0, 15.0, 18.0])
@pytest.mark.parametrize("form", ["plain", "cap", "bias"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_tails(monkeypatch, name, form, above):
    nq, L, page, Hq, heads, d = SHAPES[name]
    q, kc, vc, table = inputs(nq, L, page, Hq, heads, d, above)
    seq = torch.zeros(nq, dtype=torch.int32, device="cuda")
    length = torch.arange(L - nq + 1, L + 1, dtype=torch.int32, device="cuda")
    kw = dict(table=table, cap=200.0 if form == "cap" else 0.0, slopes=torch.full((Hq,), 1e-4, device="cuda") if form == "bias" else None)
    monkeypatch.setattr(A, "one_query", attend_bounds.one_query)
    got = M.attend(q, kc, vc, seq, length, want_lse=True, **kw)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, seq, length, **kw), f"{name} {form} {above}")


@pytest.mark.parametrize("T", [3, 280])
def test_selected(monkeypatch, T):
    q, kc, vc, table = inputs(T, 700, 16, 64, 1, 64, 17.0)
    g = torch.Generator().manual_seed(72)
    idx = torch.stack([torch.cat([torch.zeros(1, dtype=torch.int64), 1 + torch.randperm(699, generator=g)[:299]]) for _ in range(T)])
    idx = idx.to(torch.int32).cuda()
    seq = torch.zeros(T, dtype=torch.int32, device="cuda")
    length = torch.full_like(seq, 700)
    monkeypatch.setattr(A, "one_query", attend_bounds.one_query)
    got = M.attend_selected(q, kc, vc, idx, seq, length, table=table, want_lse=True)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, seq, length, table=table, idx=idx), f"selected {T}")


def test_shared(monkeypatch):
    """The heavy key in the prefix, the light ones behind it and in the own parts."""
    q, kc, vc, table = inputs(4, 320, 16, 8, 2, 64, 16.0)
    seq = torch.arange(4, dtype=torch.int32, device="cuda")
    own = table[0, 16:].view(4, 1).contiguous()
    pre, plen = torch.zeros_like(seq), torch.tensor([250], dtype=torch.int32, device="cuda")
    length = torch.tensor([16, 1, 0, 9], dtype=torch.int32, device="cuda")
    kw = dict(table=own, pre_table=table[:, :16].contiguous())
    monkeypatch.setattr(A, "one_query", attend_bounds.one_query)
    got = M.attend_shared(q, kc, vc, seq, length, pre, plen, want_lse=True, **kw)
    torch.cuda.synchronize()
    A.check(got, A.attend(q, kc, vc, seq, length, pre=pre, pre_len=plen, **kw), "shared")


@pytest.mark.parametrize("size", [30.0, 300.0, 3000.0])
@pytest.mark.parametrize("nq", [1, 6, 270])
def test_huge_scores_stay_finite(nq, size):
    """Scores up to some 1e7: the weight of the largest stays within fp16."""
    g = torch.Generator().manual_seed(73)
    kc, vc = ((torch.randn(1, 300, 1, 128, generator=g) * (size if i == 0 else 1.0)).to(FP).cuda() for i in range(2))
    q = (torch.randn(nq, 8, 128, generator=g) * size).to(FP).cuda()
    seq = torch.zeros(nq, dtype=torch.int32, device="cuda")
    length = torch.arange(300 - nq + 1, 301, dtype=torch.int32, device="cuda")
    out, lse = M.attend(q, kc, vc, seq, length, want_lse=True)
    torch.cuda.synchronize()
    want = A.attend(q, kc, vc, seq, length)
    assert bool(torch.isfinite(out).all())
    assert bool((out.abs().amax(-1) > 0).all())
    # the maximum of a row: scores of 128 products, and lse itself, in fp32
    far = (lse.cpu().double() - want[1]).abs()
    assert bool((far <= want[3]).all()), float((far / want[3]).max())
