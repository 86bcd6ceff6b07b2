"""Values that are not finite at visible keys whose weights vanish: they reach
the row whichever workgroup took them, also where the parts of several are joined."""
import math

import pytest
import torch

import attend_oracle as A
from routed_token_indexer_amd import _lib as M

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def caches(g, rows, L, heads, d, dtype):
    return tuple(torch.randn(rows, L, heads, d, generator=g).to(dtype).cuda() for _ in range(2))


def rest_is(got, want, cols, label):
    """Everything but the columns ``cols`` of the outputs, and lse, as without the values in question."""
    out = got[0].clone()
    for i in cols:
        out[..., i] = want[0][..., i].to(out.dtype).cuda()
    A.check((out, got[1]), want, label)


@pytest.mark.parametrize("bad", [37, 5000, 16383])
@pytest.mark.parametrize("Hq,d,dtype", [(4, 64, BF), (4, 128, FP), (24, 64, BF), (24, 256, FP), (48, 128, BF), (100, 256, BF)])
def test_far_keys_under_steep_slopes(Hq, d, dtype, bad):
    """One row cut into many parts; the weights of all but the nearest keys are zero in fp32."""
    g = torch.Generator().manual_seed(61)
    L = 16384
    kc, vc = caches(g, 1, L, 1, d, dtype)
    q = torch.randn(1, Hq, d, generator=g).to(dtype).cuda()
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    length = one + L
    kw = dict(slopes=torch.linspace(1.0, 4.0, Hq).cuda())
    want = A.attend(q, kc, vc, one, length, **kw)
    clean = M.attend(q, kc, vc, one, length, want_lse=True, **kw)
    vc[0, bad, 0, 3], vc[0, bad, 0, 7], vc[0, bad, 0, 9] = math.nan, math.inf, -math.inf
    got = M.attend(q, kc, vc, one, length, want_lse=True, **kw)
    torch.cuda.synchronize()
    A.check(clean, want, "before")
    assert bool(torch.isnan(got[0][..., 3]).all())
    assert not bool(torch.isfinite(got[0][..., [7, 9]]).any())
    rest_is(got, want, (3, 7, 9), f"token {bad}")


@pytest.mark.parametrize("far,near", [(200, 15900), (14000, 13000)])
def test_one_dominant_key(far, near):
    """No bias: one key's score is hundreds above all others."""
    g = torch.Generator().manual_seed(62)
    L, d = 20000, 128
    kc, vc = caches(g, 2, L, 2, d, BF)
    q = torch.randn(2, 8, d, generator=g).to(BF).cuda()
    q[..., 0] = 40.0
    kc[..., 0] = -1.0
    kc[:, 15000, :, 0] = 100.0                               # scores of 350 against -3.5
    seq = torch.arange(2, dtype=torch.int32, device="cuda")
    length = torch.tensor([L, 16000], dtype=torch.int32, device="cuda")
    want = A.attend(q, kc, vc, seq, length)
    vc[0, far, 1, 5] = math.nan                              # second kv head of the first sequence
    vc[1, near, 0, 6] = math.inf
    out, lse = M.attend(q, kc, vc, seq, length, want_lse=True)
    torch.cuda.synchronize()
    assert bool(torch.isnan(out[0, 4:, 5]).all()) and not bool(torch.isfinite(out[1, :4, 6]).any())
    assert bool(torch.isfinite(out[0, :4]).all()) and bool(torch.isfinite(out[1, 4:]).all())
    out = out.clone()
    out[0, 4:, 5], out[1, :4, 6] = want[0][0, 4:, 5].to(BF).cuda(), want[0][1, :4, 6].to(BF).cuda()
    A.check((out, lse), want, "dominant key")


@pytest.mark.parametrize("P,L", [(9000, 50), (60, 9000), (40, 30)])
def test_shared_prefix(P, L):
    """A NaN in a prefix whose weights vanish behind the own keys, and the other way round."""
    g = torch.Generator().manual_seed(63)
    rows, d = max(P, L), 64
    kc, vc = caches(g, 4, rows, 1, d, BF)                   # rows 0: the prefix, 1 .. 3: the sequences
    q = torch.randn(3, 4, d, generator=g).to(BF).cuda()
    seq = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    length, pre = torch.full_like(seq, L), torch.zeros_like(seq)
    plen = torch.tensor([P], dtype=torch.int32, device="cuda")
    for own in (False, True):
        pos = torch.full_like(seq, 0 if own else P + L - 1)  # the nearest keys: of the prefix, or the own ones
        kw = dict(slopes=torch.full((4,), 20.0, device="cuda"), q_pos=pos)
        v2 = vc.clone()
        if own:
            v2[2, L - 1, 0, 11] = math.nan
        else:
            v2[0, 1, 0, 11] = math.nan
        want = A.attend(q, kc, vc, seq, length, pre=pre, pre_len=plen, **kw)
        out, lse = M.attend_shared(q, kc, v2, seq, length, pre, plen, want_lse=True, **kw)
        torch.cuda.synchronize()
        hit = torch.tensor([False, True, False] if own else [True] * 3)
        assert torch.equal(torch.isnan(out[..., 11]).all(1).cpu(), hit) and bool(torch.isfinite(out[~hit.cuda()]).all())
        rest_is((out, lse), want, (11,), f"own {own}")
