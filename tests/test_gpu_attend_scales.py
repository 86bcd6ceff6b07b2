"""Scales from one end of the documented range to the other, and keys whose scores
are far apart or equal at any size: the formula's weights, of which the largest is
one, whatever the exponent that it is taken from."""
import pytest
import torch

import attend_oracle as A
from routed_token_indexer_amd import _lib as M

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16

# nq, Hq, heads, d: tiles of 16, 32, 64 and 128 rows
TILES = [(1, 8, 1, 64), (1, 24, 1, 128), (3, 8, 1, 256), (6, 8, 1, 64), (7, 8, 1, 128), (6, 8, 1, 256), (40, 4, 1, 64), (270, 2, 1, 128),
         (270, 2, 1, 256)]


def whole_numbers(g, *shape):
    """Values whose dot products are exact in fp32, and many of them equal."""
    return torch.randint(-2, 3, shape, generator=g).float()


@pytest.mark.parametrize("scale,size", [(1e-30, 1), (1e-10, 1), (1.0, 1), (1e3, 1), (1e4, 1), (1e4, 4), (1e4, 8)])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("tile", TILES, ids=[f"{t[0]}x{t[1]}-d{t[3]}" for t in TILES])
def test_scales(tile, dtype, scale, size):
    nq, Hq, heads, d = tile
    if size == 8:
        scale *= 64 / d          # products grow with d: up to 5e7 at each
    g = torch.Generator().manual_seed(91)
    L, page = 300 + nq, 32
    cols = -(-L // page)
    table = torch.randperm(cols, generator=g).view(1, cols).to(torch.int32).cuda()
    kc = (whole_numbers(g, cols, page, heads, d) * size).to(dtype).cuda()
    vc = torch.randn(cols, page, heads, d, generator=g).to(dtype).cuda()
    q = (whole_numbers(g, nq, Hq, d) * size).to(dtype).cuda()
    seq = torch.zeros(nq, dtype=torch.int32, device="cuda")
    length = torch.arange(L - nq + 1, L + 1, dtype=torch.int32, device="cuda")
    for cap in (0.0, 30.0):
        kw = dict(table=table, scale=scale, cap=cap)
        got = M.attend(q, kc, vc, seq, length, want_lse=True, **kw)
        torch.cuda.synchronize()
        if not cap and scale >= 1e3:
            # the products are exact, so the only scores that count are those that equal the maximum: their mean
            k, v = (A.gather_rows(x.cpu(), table.cpu(), 0, torch.arange(L)) for x in (kc, vc))
            x = (q.cpu().double() @ k[:, 0].T)
            x[torch.arange(L)[None, None, :] >= length.cpu()[:, None, None].expand(nq, Hq, 1)] = -1e9
            top = x == x.amax(-1, keepdim=True)
            assert float(x.amax()) * scale < 5e7
            n = top.sum(-1).double()
            out, mag = (top.double() @ v[:, 0]) / n[..., None], (top.double() @ v[:, 0].abs()) / n[..., None]
            lse = x.amax(-1) * scale + n.log()
            # equal weights, each rounded to 16 bits as the result is; sums of few terms
            u = A.step(dtype)
            tol = 2 * u * mag + 40 * A.E * mag + (2.0 ** -25 if dtype == FP else 0.0)
            A.check(got, (out, lse, tol, 16 * A.E * lse.abs() + 1e-5), f"scale {scale}")
        else:
            A.check(got, A.attend(q, kc, vc, seq, length, **kw), f"scale {scale} cap {cap}")


@pytest.mark.parametrize("dtype", [BF, FP])
def test_scales_in_parts(dtype):
    """One long row cut into parts, equal maxima in several of them; selected tokens and a prefix."""
    g = torch.Generator().manual_seed(92)
    L, d = 9000, 64
    kc, vc = whole_numbers(g, 2, L, 1, d).to(dtype).cuda(), torch.randn(2, L, 1, d, generator=g).to(dtype).cuda()
    q = whole_numbers(g, 2, 4, d).to(dtype).cuda()
    kc[:, 100], kc[:, 4500], kc[:, 8999] = 4.0, 4.0, 4.0
    q = q.abs() + 1
    want = vc[:, [100, 4500, 8999], 0].double().mean(1)[:, None].cpu()
    mag = vc[:, [100, 4500, 8999], 0].double().abs().mean(1)[:, None].cpu()
    tol = 3 * A.step(dtype) * mag + (2.0 ** -25 if dtype == FP else 0.0)
    seq = torch.arange(2, dtype=torch.int32, device="cuda")
    length = torch.full_like(seq, L)
    idx = torch.randperm(L, generator=g).to(torch.int32).cuda().expand(2, L).contiguous()
    for scale in (10.0, 1e3, 1e4):
        outs = [M.attend(q, kc, vc, seq, length, scale=scale)[0], M.attend_selected(q, kc, vc, idx, seq, length, scale=scale)[0]]
        # (the maxima all in the prefix, or all in the own part: the join goes by log-sums, which fp32 rounds)
        args = dict(scale=scale)
        outs += [M.attend_shared(q, kc, vc, seq, length, 1 - seq, torch.full_like(seq, 90), **args)[0],
                 M.attend_shared(q, kc, vc, 1 - seq, torch.full_like(seq, 90), seq, length, **args)[0]]
        torch.cuda.synchronize()
        for o in outs:
            assert bool(((o.cpu().double() - want).abs() <= tol).all()), scale
