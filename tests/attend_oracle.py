"""Plain fp64 forms of the cache append and of the attention operators, and how
far a kernel may be from them.

The bound of an attention output sums what each step may lose (u is half a step
of the 16-bit type, e = 2^-24 half a step of fp32, n the visible keys):
  - scores: a dot product of d terms summed in fp32 in any order loses at most
    d e sum|q k| scale; the scale, cap, bias and the reference maximum are a
    handful of further fp32 operations on values of at most |x| + |slope dist| +
    |m|. An error dx of a score is a relative error of its weight, and so is one
    of the maximum it is taken against; exp2 itself is good to 2^-22.
  - weights: rounded to 16 bits for the product (u each; fp16 has no more than
    2^-25 absolute below its normal range, against a largest weight of one);
  - sums of n products in fp32: n e each, of the weights and of the outputs;
  - the result is rounded once (u |o|, fp16 2^-25 below its normal range).
"""
import math

import torch

E = 2.0 ** -24


def step(dtype):
    return torch.finfo(dtype).eps / 2


def gather_rows(cache, table, seq, ids):
    """Rows ``ids`` of sequence ``seq``, [n, heads, d] fp64; NaN rows where the table has no page."""
    page = cache.shape[1]
    if table is None:
        return cache[seq, ids].double()
    p = table[seq, ids // page].long()
    ok = (p >= 0) & (p < cache.shape[0])
    rows = cache[p.clamp(0, cache.shape[0] - 1), ids % page].double()
    rows[~ok] = math.nan
    return rows


def one_query(q, k, v, scale, cap, slopes, dist, dtype):
    """q [Hq, d], k/v [n, heads, d] (visible tokens), dist [n] or None: out, lse and their bounds."""
    Hq, d = q.shape
    n, heads = k.shape[0], k.shape[1]
    if n == 0:
        z = torch.zeros(Hq, d, dtype=torch.float64)
        return z, torch.full((Hq,), -math.inf, dtype=torch.float64), z.clone(), torch.zeros(Hq, dtype=torch.float64)
    g = Hq // heads
    kh, vh = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)      # [n, Hq, d]
    x = torch.einsum("hd,nhd->hn", q, kh) * scale
    mag = torch.einsum("hd,nhd->hn", q.abs(), kh.abs()) * scale
    dx = (d + 2) * E * mag
    if cap:
        x = cap * torch.tanh(x / cap)
        # tanh = 1 - 2 / (1 + t), t = exp2(..): the exponent's rounding moves it by at most |y| (1 - tanh^2) e < 0.45 e,
        # exp2 (2 e) by 2 t / (1 + t)^2 2 e <= e, the sum (e) and the reciprocal (2 e) by 2 / (1 + t) 3 e <= 6 e, the
        # last difference by e: under 9 e of one, times the cap. Caps above 256 take y P(y^2) up to |y| = 0.35, fitted to
        # e and rounded in each of its steps: under 9 e of the value.
        dx = dx + 9 * E * torch.where((x.abs() > 0.3 * cap) | (cap <= 256), torch.full_like(x, float(cap)), x.abs())
    if slopes is not None:
        b = slopes.double()[:, None] * dist[None, :]
        x = x - b
        dx = dx + 4 * E * b.abs()
    m = x.amax(1, keepdim=True)
    dx = dx + 4 * E * (x.abs() + m.abs()) + 2.0 ** -22
    p = torch.exp(x - m)
    L = p.sum(1)
    out = torch.einsum("hn,nhd->hd", p, vh) / L[:, None]
    lse = m[:, 0] + torch.log(L)
    u = step(dtype)
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    # the sum's relative error, from the weights' and its own rounding
    dl = (p * dx).sum(1) / L + dx.amax(1) * 0 + n * E
    absv = torch.einsum("hn,nhd->hd", p * (u + dx + dl[:, None] + (n + 8) * E) + tiny, vh.abs()) / L[:, None]
    # a part that another workgroup joins carries a few more fp32 roundings
    tol = u * out.abs() + absv * (1 + u) + tiny + 16 * E * out.abs()
    return out, lse, tol, dl + dx.amax(1) + 8 * E * (1 + lse.abs())


def attend(q, k_cache, v_cache, q_seq, q_len, table=None, q_start=None, q_pos=None, scale=None, cap=0.0, slopes=None,
           idx=None, pre=None, pre_len=None, pre_table=None):
    """All queries on the CPU; returns out, lse, tol, tol_lse (fp64)."""
    cpu = lambda t: None if t is None else t.detach().cpu()   # noqa: E731
    q, kc, vc, q_seq, q_len, table, q_start, q_pos, slopes, idx, pre, pre_len, pre_table = map(
        cpu, (q, k_cache, v_cache, q_seq, q_len, table, q_start, q_pos, slopes, idx, pre, pre_len, pre_table))
    if kc.dim() == 3:
        kc, vc = kc[:, :, None], vc[:, :, None]
    T, Hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    page = kc.shape[1]
    nseq = kc.shape[0] if table is None else table.shape[0]
    Lmax = page * (1 if table is None else table.shape[1])
    outs = []
    for t in range(T):
        n = int(q_seq[t])
        ok = 0 <= n < nseq
        end = min(max(int(q_len[t]), 0), Lmax) if ok else 0
        begin = 0 if q_start is None else min(max(int(q_start[t]), 0), end)
        if idx is not None:
            ids = idx[t].long()
            ids = ids[(ids >= 0) & (ids < end)] if ok else ids[:0]
        else:
            ids = torch.arange(begin, end)
        k, v = (gather_rows(kc, table, n, ids), gather_rows(vc, table, n, ids)) if ok else (kc[:0, 0].double(), vc[:0, 0].double())
        at = ids
        plen = 0
        if pre is not None and ok:
            i = int(pre[t])
            if 0 <= i < len(pre_len):
                most = page * (1 if pre_table is None else pre_table.shape[1])
                plen = min(max(int(pre_len[i]), 0), most)
                ahead = torch.arange(plen)
                k = torch.cat([gather_rows(kc, pre_table, i, ahead), k])
                v = torch.cat([gather_rows(vc, pre_table, i, ahead), v])
                at = torch.cat([ahead, at + plen])
        if table is not None or pre_table is not None:      # tokens without a page are not visible
            have = ~_no_page(kc, table, n, ids, ok)
            if plen:
                have = torch.cat([~_no_page(kc, pre_table, i, ahead, True), have])
            k, v, at = k[have], v[have], at[have]
        dist = None
        if slopes is not None:
            pos = int(q_pos[t]) if q_pos is not None else plen + int(q_len[t]) - 1
            dist = (pos - at).abs().double()
        outs.append(one_query(q[t].double(), k, v, scale, cap, slopes, dist, q.dtype))
    return tuple(torch.stack([o[i] for o in outs]) if outs else torch.zeros(0) for i in range(4))


def _no_page(cache, table, seq, ids, ok):
    if not ok or table is None:
        return torch.zeros(len(ids), dtype=torch.bool)
    p = table[seq, ids // cache.shape[1]]
    return (p < 0) | (p >= cache.shape[0])


def check(got, want, label=""):
    """Kernel outputs (out, lse) against the oracle's (out, lse, tol, tol_lse)."""
    out, lse = got
    o, l, tol, tol_l = want
    err = (out.detach().cpu().double() - o).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), f"{label}: {int(bad.sum())} outputs off, worst {float((err / tol.clamp(min=1e-30)).max()):.3g} of the bound"
    if lse is not None:
        lse = lse.detach().cpu().double()
        none = l == -math.inf
        assert torch.equal(lse == -math.inf, none), f"{label}: rows without a key"
        err = (lse - l).abs()[~none]
        assert bool((err <= tol_l[~none]).all()), f"{label}: lse off, worst {float((err / tol_l[~none]).max()):.3g} of the bound"


def rotate(x, cos_sin, pos, interleaved):
    """x [N, heads, d] fp64 turned by rows ``pos`` of cos_sin [P, rot]."""
    rot = cos_sin.shape[1]
    h = rot // 2
    c, s = cos_sin[pos, None, :h].double(), cos_sin[pos, None, h:].double()
    y = x.double().clone()
    a, b = (y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()) if interleaved else (y[..., :h].clone(), y[..., h:rot].clone())
    ra, rb = a * c - b * s, b * c + a * s
    # two products and a sum in fp32, then one rounding to the type
    bound = 3 * E * (a.abs() * c.abs() + b.abs() * s.abs()), 3 * E * (b.abs() * c.abs() + a.abs() * s.abs())
    tol = torch.zeros_like(y)
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = ra, rb
        tol[..., 0:rot:2], tol[..., 1:rot:2] = bound
    else:
        y[..., :h], y[..., h:rot] = ra, rb
        tol[..., :h], tol[..., h:rot] = bound
    u = step(x.dtype)
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 0.0
    turned = torch.zeros_like(y, dtype=torch.bool)
    turned[..., :rot] = True
    return y, torch.where(turned, tol * (1 + u) + u * y.abs() + tiny, torch.zeros_like(y))
