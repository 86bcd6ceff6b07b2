"""Plain fp64 forms of accumulated attention weight, eviction and sampling, and how far
a kernel may be from them.

A cached token's sum of weights e^(x - lse) (E = 2^-24, half a step of fp32):
  - a score loses what attend_oracle.py derives: at most d E sum|q k| scale in the dot
    product, a handful of further fp32 operations on values of the size of |x|, the
    bias and |lse|, 9 E of one times the cap (of the value for caps above 256). An error of
    the score is a relative error of its weight, and exp2 is good to 2^-22;
  - the sum of n weights, in any order and joined from parts, n E of itself; one more
    rounding where the earlier sum is added.
Eviction only compares and copies: no tolerance. Sampling compares sums of weights that
are multiples of 2^-42 of the largest: V 2^-43 of it, and the fp64 oracle's own V 2^-52
of the sum, so a token is wrong unless a comparison is nearer than that.
"""
import math

import torch

import attend_oracle as A

E = A.E


def mass(q, k_cache, lse, q_seq, q_len, table=None, q_start=None, q_pos=None, scale=None, cap=0.0, slopes=None, before=None,
         lists=None):
    """Sums [nseq, lists, tokens] and their bound, fp64 on the CPU."""
    cpu = lambda t: None if t is None else t.detach().cpu()   # noqa: E731
    q, kc, lse, q_seq, q_len, table, q_start, q_pos, slopes, before = map(
        cpu, (q, k_cache, lse, q_seq, q_len, table, q_start, q_pos, slopes, before))
    if kc.dim() == 3:
        kc = kc[:, :, None]
    T, Hq, d = q.shape
    heads, page = kc.shape[2], kc.shape[1]
    scale = d ** -0.5 if scale is None else scale
    nseq = kc.shape[0] if table is None else table.shape[0]
    L = page * (1 if table is None else table.shape[1])
    G, g = lists or heads, Hq // heads
    out = torch.zeros(nseq, heads, L, dtype=torch.float64)
    tol = torch.zeros_like(out)
    count = torch.zeros_like(out)
    for t in range(T):
        n = int(q_seq[t])
        if not 0 <= n < nseq:
            continue
        end = min(max(int(q_len[t]), 0), L)
        begin = 0 if q_start is None else max(int(q_start[t]), 0)
        ids = torch.arange(begin, max(end, begin))
        ids = ids[~A._no_page(kc, table, n, ids, True)]
        if not len(ids):
            continue
        k = A.gather_rows(kc, table, n, ids).repeat_interleave(g, 1)      # [n, Hq, d]
        x = torch.einsum("hd,nhd->hn", q[t].double(), k) * scale
        dx = (d + 2) * E * torch.einsum("hd,nhd->hn", q[t].double().abs(), k.abs()) * scale
        if cap:
            x = cap * torch.tanh(x / cap)
            dx = dx + 9 * E * torch.where((x.abs() > 0.3 * cap) | (cap <= 256), torch.full_like(x, float(cap)), x.abs())
        if slopes is not None:
            pos = int(q_pos[t]) if q_pos is not None else int(q_len[t]) - 1
            b = slopes.double()[:, None] * (pos - ids).abs().double()
            x = x - b
            dx = dx + 4 * E * b.abs()
        l = lse[t].double()[:, None]
        none = l == -math.inf
        dx = torch.where(none, 0.0, dx + 4 * E * (x.abs() + l.abs()) + 2.0 ** -22)
        w = torch.where(none, 0.0, torch.exp(x - l)).view(heads, g, -1)
        out[n][:, ids] += w.sum(1)
        tol[n][:, ids] += (w * torch.expm1(dx.view(heads, g, -1))).sum(1)
        count[n][:, ids] += g
    if G == 1:
        out, tol, count = (x.sum(1, keepdim=True) for x in (out, tol, count))
    tol = tol + (count + 16 + heads) * E * out + 2.0 ** -126
    if before is not None:
        out = out + before.double()
        tol = tol + E * out.abs()
    return out, tol


def check_mass(got, want, label=""):
    g, (w, tol) = got.detach().cpu().double(), want
    assert g.shape == w.shape
    bad = ~((g - w).abs() <= tol) & ~(g.isnan() & w.isnan())
    assert not bool(bad.any()), f"{label}: {int(bad.sum())} sums off, worst {float(((g - w).abs() / tol).nan_to_num(9e9).max()):.3g} of the bound"


def evict(mass, pos, lens, budget, sinks, recent):
    """new_len, src, mass_out, pos_out on the CPU, by sorting the rows of each list."""
    mass, lens = mass.cpu(), lens.cpu()
    nseq, G, L = mass.shape
    pos = torch.arange(L, dtype=torch.int32).expand(nseq, G, L) if pos is None else pos.cpu()
    src = torch.full((nseq, G, budget), -1, dtype=torch.int32)
    mo, po = torch.zeros_like(mass), torch.full((nseq, G, L), -1, dtype=torch.int32)
    size = [min(max(int(v), 0), L) for v in lens]
    for n in range(nseq):
        ln, sz = size[n], min(size[n], budget)
        for g in range(G):
            m, p = mass[n, g, :ln].tolist(), pos[n, g, :ln].tolist()
            newest = max(p, default=0)

            def rank(i):
                if p[i] < sinks or p[i] > newest - recent:
                    return 0, 0.0, i
                return (1, 0.0, i) if m[i] != m[i] else (2, -m[i], i)
            order = sorted(range(ln), key=rank)
            kept = set(order[:sz])
            holes = [i for i in range(sz) if i not in kept]
            movers = sorted(i for i in kept if i >= sz)
            assert len(holes) == len(movers)
            row = list(range(sz))
            for h, v in zip(holes, movers):
                row[h] = v
            row = torch.tensor(row, dtype=torch.long)
            src[n, g, :sz] = row.int()
            mo[n, g, :sz], po[n, g, :sz] = mass[n, g][row], pos[n, g][row]
    return torch.tensor([min(s, budget) for s in size], dtype=torch.int32), src, mo, po


def move(cache, src, table=None):
    """The cache after the moves; source rows as they were before."""
    x = cache.cpu().clone()
    if x.dim() == 3:
        return move(x[:, :, None], src, table)[:, :, 0]
    old, src = x.clone(), src.cpu()
    table = None if table is None else table.cpu()
    page, L = x.shape[1], x.shape[1] * (1 if table is None else table.shape[1])

    def at(n, s):
        if table is None:
            return n, s
        p = int(table[n, s // page])
        return (p, s % page) if 0 <= p < x.shape[0] else None
    for n in range(src.shape[0]):
        for g in range(src.shape[1]):
            heads = slice(None) if src.shape[1] == 1 else slice(g, g + 1)
            for i in range(min(src.shape[2], L)):
                s = int(src[n, g, i])
                if 0 <= s < L and s != i and at(n, s) and at(n, i):
                    x[at(n, i)][heads] = old[at(n, s)][heads]
    return x


def bits(x):
    return x.detach().cpu().contiguous().view({2: torch.int16, 4: torch.int32}[x.element_size()])


def sample_row(l, u, t=1.0, k=0, p=1.0, m=0.0):
    """(tokens that may be drawn, {token: log-probability}): one token unless a comparison is too near to tell."""
    l = l.detach().cpu().double()
    V = len(l)
    l = torch.where(l.isnan(), torch.full_like(l, -math.inf), l)
    top = float(l.max())
    if top == -math.inf:
        return {-1}, {-1: -math.inf}
    if not t > 0:
        i = int((l == top).nonzero()[0])
        return {i}, {i: 0.0}
    x = torch.where(l == top, torch.zeros_like(l), (l - top) / t).nan_to_num(nan=-math.inf)
    w = torch.exp(x)
    order = torch.argsort(l, descending=True, stable=True)
    near = V * 2.0 ** -43 + V * 2.0 ** -52

    def keep_sizes(k, p, m):
        """Prefixes of the order that the filters may leave."""
        n = k if 0 < k < V else V
        if m > 0:
            n = min(n, int((w[order] >= min(m, 1.0)).sum()))
        sizes = {n}
        if p < 1:
            run = torch.cumsum(w[order[:n]], 0)
            goal = max(p, 0.0) * float(run[-1])
            sizes = set()
            for off in (-near, near):
                sizes.add(min(n, int((run < goal + off * max(1.0, float(run[-1]))).sum()) + 1))
            # exact sums (equal weights): no doubt
            if bool((w[order[:n]] == w[order[0]]).all()):
                sizes = {max(1, min(n, math.ceil(max(p, 0.0) * n)))}
        return sizes
    u = 0.0 if not u > 0 else min(u, 1.0)
    may, logs = set(), {}
    for n in keep_sizes(k, p, m):
        ids = order[:n].sort().values
        run = torch.cumsum(w[ids], 0)
        total = float(run[-1])
        # equal weights: the sums are whole numbers times one weight, and nothing is in doubt
        for off in (0.0,) if bool((w[ids] == w[ids[0]]).all()) else (-near, near):
            i = int((run <= u * total + off * max(1.0, total)).sum())
            alive = (w[ids] > 2.0 ** -43).nonzero()
            i = min(i, int(alive[-1]))
            i = int(alive[(alive >= i)][0]) if bool((alive >= i).any()) else i
            tok = int(ids[i])
            may.add(tok)
            logs[tok] = float(x[tok]) - math.log(total)
    return may, logs
