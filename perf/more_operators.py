"""Measured cases of what bounds a cache and what ends a decode step.

Four operators, each in a plain form (elementary torch operations) and as the
library's own call:

  mass    how much attention weight each cached token got, summed over queries and heads
  evict   keep the tokens of most weight and make them the first rows of the cache, in place
  move    the same moves in another cache
  sample  the next tokens from logits: temperature, top-k, min-p, top-p, given random numbers

Eviction fills the rows of dropped tokens with the kept tokens from behind the
budget, so no row that is read is written, and a second pass over the same
state gives the same.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a small decode step of short chats with capped scores: latency counts
        dict(name="mass_decode_short", op="mass", nseq=8, nq=1, L=1500, page=16, Hq=32, Hkv=8, d=64, mask="causal",
             cap=30.0, bias=False, shared=False, type="fp16", layout="token"),
        # a decode step over long, uneven prefixes: bound by the keys' bytes
        dict(name="mass_decode_long", op="mass", nseq=8, nq=1, L=32768, page=64, Hq=64, Hkv=8, d=128, mask="causal",
             cap=0.0, bias=False, shared=False, type="bf16", layout="token"),
        # the last 64 positions of two long prompts say what of the prompt is kept
        dict(name="mass_window", op="mass", nseq=2, nq=64, L=32768, page=64, Hq=64, Hkv=8, d=128, mask="causal",
             cap=0.0, bias=False, shared=False, type="bf16", layout="token"),
        # every position of a prompt: bound by the matrix cores and the exponentials
        dict(name="mass_prompt", op="mass", nseq=1, nq=8192, L=8192, page=64, Hq=64, Hkv=8, d=128, mask="causal",
             cap=0.0, bias=False, shared=False, type="bf16", layout="token"),
        # packed documents with a distance bias and wide heads, one sum over all heads
        dict(name="mass_documents", op="mass", nseq=2, nq=2000, L=2000, page=48, Hq=16, Hkv=4, d=256, mask="documents",
             cap=0.0, bias=True, shared=True, type="fp16", layout="head"),
        # a decode batch that is 64 tokens over its budget, one choice for all heads
        dict(name="evict_step", op="evict", nseq=64, L=2112, even=True, budget=2048, sinks=4, recent=128, page=64, Hkv=8,
             d=128, shared=True, order=False, values=True, type="bf16", layout="token"),
        # long prompts cut to a short cache, each head by its own weights
        dict(name="evict_prompt", op="evict", nseq=4, L=32768, even=False, budget=2048, sinks=4, recent=64, page=64,
             Hkv=8, d=128, shared=False, order=True, values=True, type="bf16", layout="token"),
        # the indexer's keys (one head, contiguous rows, no values) follow
        dict(name="move_index_keys", op="move", nseq=4, L=32768, even=False, budget=4096, sinks=4, recent=64, page=0,
             Hkv=1, d=128, shared=True, order=True, values=False, type="bf16", layout="token"),
        # another layer's cache follows
        dict(name="move_layer", op="move", nseq=8, L=32768, even=False, budget=8192, sinks=4, recent=64, page=64, Hkv=8,
             d=128, shared=True, order=True, values=True, type="fp16", layout="head"),
        # four chats, all filters
        dict(name="sample_small", op="sample", T=4, V=32000, type="bf16", filters="all", pad=0),
        # a batch whose requests ask for different things, fp32 logits
        dict(name="sample_batch", op="sample", T=64, V=128000, type="fp32", filters="mixed", pad=0),
        # a large batch, temperature and top-p, rows of a padded matrix product
        dict(name="sample_large", op="sample", T=256, V=151643, type="bf16", filters="top_p", pad=293),
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b + 0.49)))))))


def draw(rng):
    op = rng.choice(["mass", "mass", "evict", "move", "sample"])
    kind = rng.choice(["bf16", "fp16"])
    if op == "sample":
        V = _log(rng, 2, 200000)
        return dict(op=op, T=_log(rng, 1, max(1, min(512, 38000000 // V))), V=V, type=rng.choice(["bf16", "fp16", "fp32"]),
                    filters=rng.choice(["none", "top_k", "top_p", "min_p", "all", "mixed"]), pad=rng.choice([0, 0, 5, 64]))
    Hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, page=rng.choice([1, 16, 24, 48, 64, 128, 256]), Hkv=Hkv, type=kind, layout=rng.choice(["token", "head"]),
             shared=rng.random() < 0.4)
    if op == "mass":
        c["Hq"] = Hkv * rng.choice([1, 2, 3, 4, 7, 8, 16])
        c["d"] = d = rng.choice([64, 128, 256])
        c["cap"] = rng.choice([0.0, 0.0, 20.0, 50.0])
        c["bias"] = rng.random() < 0.3
        c["mask"] = rng.choice(["causal", "causal", "documents"])
        form = rng.choice(["step", "step", "window", "prompt"])
        if form == "step":
            c["nseq"], c["nq"] = _log(rng, 1, 48), rng.choice([1, 1, 2, 5])
            c["L"] = _log(rng, max(8, c["nq"]), min(60000, (1 << 27) // (c["nseq"] * Hkv * d)))
        elif form == "window":
            c["nseq"], c["nq"] = rng.choice([1, 2, 3, 5]), rng.choice([8, 16, 33, 64])
            c["L"] = _log(rng, c["nq"], min(40000, (1 << 27) // (c["nseq"] * Hkv * d)))
        else:
            c["nseq"] = rng.choice([1, 2, 3])
            c["nq"] = _log(rng, 65, 2500)
            c["L"] = c["nq"] + rng.choice([0, _log(rng, 1, 1000)])
        return c
    c["d"] = rng.choice([64, 96, 128, 256])
    c["nseq"] = _log(rng, 1, 64)
    c["L"] = _log(rng, 4, min(60000, (1 << 27) // (c["nseq"] * Hkv * c["d"])))
    c["even"] = rng.random() < 0.3
    c["budget"] = _log(rng, 1, c["L"])
    c["sinks"] = min(c["budget"] // 4, 4)
    c["recent"] = min(c["budget"] // 2, _log(rng, 1, 256))
    c["order"] = rng.random() < 0.5
    c["values"] = rng.random() < 0.8
    return c


# ---------------------------------------------------------------- lengths (of the case alone)
def _len_of(c, n, least):
    """Uneven lengths of a batch: the first sequence is the longest."""
    if c.get("even"):
        return c["L"]
    return max(least, min(c["L"], int(c["L"] * (1.0 - 0.75 * ((n * 0.618034) % 1.0)))))


def _intervals(c):
    """Visible interval [start, len) and position of each query, as three lists."""
    start, length, pos = [], [], []
    for n in range(c["nseq"]):
        total = _len_of(c, n, c["nq"])
        doc = max(1, total // 7)
        for i in range(c["nq"]):
            p = total - c["nq"] + i
            start.append(p // doc * doc if c["mask"] == "documents" else 0)
            length.append(p + 1)
            pos.append(p)
    return start, length, pos


# ---------------------------------------------------------------- inputs
def _cache(g, c, pages, page, dev, dt):
    """Cache tensor [pages, page, Hkv, d], stored token-major or head-major."""
    Hkv, d = c["Hkv"], c["d"]
    if c["layout"] == "head":
        return torch.randn(pages, Hkv, page, d, generator=g, device=dev, dtype=torch.float32).to(dt).permute(0, 2, 1, 3)
    return torch.randn(pages, page, Hkv, d, generator=g, device=dev, dtype=torch.float32).to(dt)


def _log_sums(s):
    """The log-sums that attention over the same keys returned."""
    c = s["case"]
    out = torch.empty(s["q"].shape[:2], device=s["q"].device)
    for h in range(c["Hkv"]):
        g = c["Hq"] // c["Hkv"]
        x = _scores(s, s["q"][:, h * g:(h + 1) * g], s["k_cache"][:, :, h:h + 1], h * g)
        out[:, h * g:(h + 1) * g] = torch.logsumexp(x, -1).permute(0, 2, 1, 3).reshape(-1, g)
    return out


def _kept(c, s, g):
    """Random moves of an eviction: [sequences, lists, budget], -1 behind the kept rows."""
    G = 1 if c["shared"] else c["Hkv"]
    mass = torch.rand(c["nseq"], G, c["L"], generator=g, device=s["lens"].device)
    kept = _chosen(mass, None, s["lens"], c["budget"], c["sinks"], c["recent"])
    return _sources(kept, s["lens"], c["budget"])


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = _TYPES[c["type"]]
    s = dict(case=c)
    if c["op"] == "sample":
        T, V = c["T"], c["V"]
        # a broad floor of tokens, and some dozens that the context makes likely
        rows = torch.randn(T, V + c["pad"], generator=g, device=dev).mul_(1.5)
        n = min(V, 60)
        at = torch.randint(0, V, (T, n), generator=g, device=dev)
        rows.scatter_add_(1, at, 9.0 - 0.12 * torch.arange(n, device=dev) + torch.randn(T, n, generator=g, device=dev))
        s["logits"] = rows.to(dt)[:, :V]
        u = lambda lo, hi: torch.rand(T, generator=g, device=dev) * (hi - lo) + lo  # noqa: E731
        s["temperature"], s["top_k"], s["top_p"], s["min_p"] = u(0.5, 1.3), None, None, None
        kind, off = c["filters"], lambda share: torch.rand(T, generator=g, device=dev) < share  # noqa: E731
        if kind in ("top_k", "all", "mixed"):
            s["top_k"] = (u(0.0, 1.0) * 80).int() + 1
        if kind in ("top_p", "all", "mixed"):
            s["top_p"] = u(0.7, 0.98)
        if kind in ("min_p", "all", "mixed"):
            s["min_p"] = u(0.0, 0.1)
        if kind == "mixed":   # each request has some of the filters; some are greedy
            s["top_k"][off(0.6)] = 0
            s["top_p"][off(0.4)] = 1.0
            s["min_p"][off(0.6)] = 0.0
            s["temperature"][off(0.1)] = 0.0
        s["u"] = torch.rand(T, generator=g, device=dev)
        return s
    ints = dict(device=dev, dtype=torch.int32)
    nseq, Hkv, d = c["nseq"], c["Hkv"], c["d"]
    page = c["page"] or c["L"]
    cols = -(-c["L"] // page)
    s["table"] = None
    if c["page"]:
        s["table"] = torch.randperm(nseq * cols, generator=g, device=dev).to(torch.int32).view(nseq, cols)
    s["k_cache"] = _cache(g, c, nseq * cols, page, dev, dt)
    G = 1 if c["shared"] else Hkv
    if c["op"] == "mass":
        T, Hq = nseq * c["nq"], c["Hq"]
        s["scale"], s["cap"] = 1.0 / math.sqrt(d), c["cap"]
        s["q"] = (1.5 * torch.randn(T, Hq, d, generator=g, device=dev, dtype=torch.float32)).to(dt)
        start, length, pos = _intervals(c)
        s["q_seq"] = torch.arange(nseq, **ints).repeat_interleave(c["nq"])
        s["q_len"] = torch.tensor(length, **ints)
        s["q_start"] = torch.tensor(start, **ints) if c["mask"] == "documents" else None
        s["q_pos"] = torch.tensor(pos, **ints) if c["bias"] else None
        s["slopes"] = (2.0 ** (-8.0 * torch.arange(1, Hq + 1, device=dev, dtype=torch.float32) / Hq)) if c["bias"] else None
        s["lse"] = _log_sums(s)
        # what earlier steps gave
        s["mass"] = torch.rand(nseq, G, cols * page, generator=g, device=dev)
        s["mass_out"] = torch.empty_like(s["mass"])
        return s
    s["v_cache"] = _cache(g, c, nseq * cols, page, dev, dt) if c["values"] else None
    lens = [_len_of(c, n, 1) for n in range(nseq)]
    s["lens"] = torch.tensor(lens, **ints)
    if c["op"] == "move":
        s["src"] = _kept(c, s, g)
        return s
    # few tokens got most of the weight
    s["mass"] = torch.randn(nseq, G, cols * page, generator=g, device=dev).mul_(2.0).exp_()
    pos = torch.arange(cols * page, **ints).expand(nseq, G, -1).clone()
    if not c["order"]:   # earlier evictions moved rows: all but the latest tokens lie anywhere
        old = max(0, min(lens) - c["recent"])
        mixed = torch.rand(nseq, G, old, generator=g, device=dev).argsort(-1)
        pos[:, :, :old] = mixed.int()
    s["pos"] = pos
    s["mass_out"], s["pos_out"] = torch.empty_like(s["mass"]), torch.empty_like(pos)
    s["src_out"], s["len_out"] = torch.empty(nseq, G, c["budget"], **ints), torch.empty(nseq, **ints)
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import routed_token_indexer_amd as misa
        if op == "mass":
            return misa.attend_mass(s["q"], s["k_cache"], s["lse"], s["q_seq"], s["q_len"], table=s["table"],
                                    q_start=s["q_start"], q_pos=s["q_pos"], scale=s["scale"], cap=s["cap"],
                                    slopes=s["slopes"], mass=s["mass"], out=s["mass_out"])
        if op == "evict":
            misa.cache_evict(s["k_cache"], s["v_cache"], s["mass"], s["lens"], c["budget"], sinks=c["sinks"],
                             recent=c["recent"], pos=s["pos"], table=s["table"], mass_out=s["mass_out"],
                             pos_out=s["pos_out"], src=s["src_out"], new_len=s["len_out"])
            return _evict_outputs(s)
        if op == "move":
            misa.cache_move(s["k_cache"], s["v_cache"], s["src"], table=s["table"])
            return _caches(s)
        return misa.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                           min_p=s["min_p"], want_logprob=True)
    return {"mass": _plain_mass, "evict": _plain_evict, "move": _plain_move, "sample": _plain_sample}[op](s)


def _caches(s):
    return [x for x in (s["k_cache"], s["v_cache"]) if x is not None]


def _evict_outputs(s):
    return [s["len_out"], s["src_out"], s["mass_out"], s["pos_out"], *_caches(s)]


def _scores(s, q, k_cache, head):
    """Masked scores of the queries' heads (the first of them is ``head``): fp32 [nseq, kv heads, nq, group, tokens]."""
    c = s["case"]
    nseq, nq, Hkv, d = c["nseq"], c["nq"], k_cache.shape[2], c["d"]
    g = q.shape[1] // Hkv
    k = k_cache if s["table"] is None else k_cache[s["table"].long()].flatten(1, 2)
    rows = q.reshape(nseq, nq, Hkv, g, d).permute(0, 2, 1, 3, 4).reshape(nseq, Hkv, nq * g, d).float()
    x = (rows @ k.transpose(1, 2).float().transpose(-1, -2)).mul_(s["scale"]).view(nseq, Hkv, nq, g, -1)
    if s["cap"]:
        x = x.div_(s["cap"]).tanh_().mul_(s["cap"])
    at = torch.arange(x.shape[-1], device=x.device)
    per = lambda v: v.view(nseq, 1, nq, 1, 1)  # noqa: E731
    if s["slopes"] is not None:
        x -= s["slopes"][head:head + q.shape[1]].view(1, Hkv, 1, g, 1) * (per(s["q_pos"]) - at).abs()
    hidden = at >= per(s["q_len"])
    if s["q_start"] is not None:
        hidden = hidden | (at < per(s["q_start"]))
    return x.masked_fill_(hidden, -math.inf)


def _plain_mass(s):
    c = s["case"]
    nseq, nq, Hkv = c["nseq"], c["nq"], c["Hkv"]
    x = _scores(s, s["q"], s["k_cache"], 0)
    x -= s["lse"].view(nseq, nq, Hkv, -1, 1).permute(0, 2, 1, 3, 4)
    got = x.exp_().sum((2, 3))
    if c["shared"]:
        got = got.sum(1, keepdim=True)
    s["mass_out"].copy_(s["mass"] + got)
    return s["mass_out"]


def _chosen(mass, pos, lens, budget, sinks, recent):
    """Which rows stay: [sequences, lists, rows]."""
    at = torch.arange(mass.shape[-1], device=mass.device, dtype=torch.int32)
    there = at < lens[:, None, None]
    p = at.expand(mass.shape) if pos is None else pos
    newest = torch.where(there, p, torch.full_like(p, -1)).amax(-1, keepdim=True)
    safe = (p < sinks) | (p > newest - recent)
    rank = torch.where(safe, torch.full_like(mass, math.inf), mass).masked_fill(~there, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :budget]
    return torch.zeros_like(there.expand(mass.shape)).scatter(-1, order, True) & there


def _sources(kept, lens, budget):
    """Row that each of the first ``budget`` rows comes from; -1 behind the kept ones."""
    rows = kept.shape[-1]
    at = torch.arange(rows, device=kept.device)
    size = lens.clamp(max=budget)[:, None, None]
    mover, hole = kept & (at >= size), ~kept & (at < size)
    # the n-th hole takes the n-th mover
    movers = torch.where(mover, at, rows).sort(-1).values
    nth = (hole.cumsum(-1) - 1).clamp(min=0)
    src = torch.where(hole, movers.gather(-1, nth), at.expand(kept.shape))
    src = torch.where(at < size, src, torch.full_like(src, -1))
    return torch.nn.functional.pad(src, (0, max(0, budget - rows)), value=-1)[..., :budget].to(torch.int32).contiguous()


def _plain_moves(s, src):
    page = s["k_cache"].shape[1]
    n, lists, row = torch.nonzero((src >= 0) & (src != torch.arange(src.shape[-1], device=src.device)), as_tuple=True)
    old = src[n, lists, row].long()
    where = (lambda t: (n, t)) if s["table"] is None else (lambda t: (s["table"][n, t // page].long(), t % page))
    (p1, r1), (p0, r0) = where(row), where(old)
    for x in _caches(s):
        if src.shape[1] == 1:
            x[p1, r1] = x[p0, r0]
        else:
            x[p1, r1, lists] = x[p0, r0, lists]


def _plain_move(s):
    _plain_moves(s, s["src"])
    return _caches(s)


def _plain_evict(s):
    c = s["case"]
    kept = _chosen(s["mass"], s["pos"], s["lens"], c["budget"], c["sinks"], c["recent"])
    src = _sources(kept, s["lens"], c["budget"])
    from_, there = src.clamp(min=0).long(), src >= 0
    s["mass_out"].zero_()
    s["pos_out"].fill_(-1)
    n = min(c["budget"], s["mass"].shape[-1])
    s["mass_out"][..., :n] = torch.where(there, s["mass"].gather(-1, from_), torch.zeros((), device=src.device))[..., :n]
    s["pos_out"][..., :n] = torch.where(there, s["pos"].gather(-1, from_), torch.full_like(src, -1))[..., :n]
    s["src_out"].copy_(src)
    s["len_out"].copy_(s["lens"].clamp(max=c["budget"]))
    _plain_moves(s, src)
    return _evict_outputs(s)


def _plain_sample(s):
    # in 64 bits: running sums over the vocabulary are compared with each other
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    warm = s["temperature"][:, None] > 0
    w = ((x - top) / torch.where(warm, s["temperature"][:, None], 1.0).double()).exp_()
    w = torch.where(warm, w, (x == top).double())
    sorted_x, order = torch.sort(x, dim=-1, descending=True, stable=True)
    p = w.gather(-1, order)
    rank = torch.arange(p.shape[-1], device=p.device)
    p = torch.where(warm | (rank == 0), p, 0.0)   # greedy: the first largest
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        p = p.masked_fill((k > 0) & (rank >= k) & warm, 0.0)
    if s["min_p"] is not None:
        p = p.masked_fill((p < s["min_p"][:, None].double()) & warm, 0.0)
    if s["top_p"] is not None:
        before = p.cumsum(-1) - p
        enough = before >= s["top_p"][:, None].double() * p.sum(-1, keepdim=True)
        p = p.masked_fill(enough & (s["top_p"][:, None] < 1) & (rank > 0) & warm, 0.0)
    w = torch.zeros_like(w).scatter_(-1, order, p)
    run_ = w.cumsum(-1)
    total = run_[:, -1:]
    token = (run_ <= s["u"][:, None].double() * total).sum(-1, keepdim=True)
    return token[:, 0].int(), (w.gather(-1, token) / total).log()[:, 0].float()


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "sample":
        return dict(bytes=c["T"] * c["V"] * (4 if c["type"] == "fp32" else 2) + 28 * c["T"], flops=2 * c["T"] * c["V"])
    G = 1 if c["shared"] else c["Hkv"]
    if c["op"] == "mass":
        start, length, _ = _intervals(c)
        nq, d = c["nq"], c["d"]
        rows = sum(max(length[n * nq:(n + 1) * nq]) - min(start[n * nq:(n + 1) * nq]) for n in range(c["nseq"]))
        page = c["page"] or c["L"]
        cols = -(-c["L"] // page) * page
        return dict(bytes=rows * c["Hkv"] * d * 2 + len(length) * c["Hq"] * (2 * d + 4) + 8 * c["nseq"] * G * cols,
                    flops=2 * d * c["Hq"] * sum(b - a for a, b in zip(start, length)))
    moved = listed_rows = rows = 0
    for n in range(c["nseq"]):
        L, B = _len_of(c, n, 1), c["budget"]
        rows += L
        listed_rows += min(L, B)
        if L > B:
            # kept tokens behind the budget: the latest ones that lie there, and of the chosen ones their share
            latest = min(c["recent"], L - B)
            free = max(1, L - c["sinks"] - c["recent"])
            moved += latest + max(0, B - c["sinks"] - c["recent"]) * max(0, L - B - latest) / free
    pairs = 2 if c["values"] else 1
    row = 2 * c["Hkv"] * c["d"] * pairs
    lists = 4 * G * listed_rows
    chosen = 0 if c["op"] == "move" else G * 8 * (rows + listed_rows)
    return dict(bytes=int(2 * moved * row + lists + chosen), flops=0)


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "sample":
        return _exact_sample(s)
    if c["op"] == "mass":
        return _exact_mass(s)
    src = s["src"] if c["op"] == "move" else None
    out = []
    if c["op"] == "evict":
        mass, pos, lens = s["mass"].cpu(), s["pos"].cpu(), s["lens"].tolist()
        new_mass, new_pos = torch.zeros_like(mass), torch.full_like(pos, -1)
        src = torch.full((*mass.shape[:2], c["budget"]), -1, dtype=torch.int32)
        size = [min(L, c["budget"]) for L in lens]
        for n, L in enumerate(lens):
            for g in range(mass.shape[1]):
                m, p = mass[n, g, :L], pos[n, g, :L]
                safe = (p < c["sinks"]) | (p > int(p.max()) - c["recent"])
                # by protection, weight and row: the last key is sorted first
                by = torch.argsort(m, descending=True, stable=True)
                by = by[torch.argsort(safe[by].int(), descending=True, stable=True)][:size[n]]
                stay = torch.zeros(L, dtype=torch.bool)
                stay[by] = True
                rows = torch.arange(size[n])
                rows[~stay[:size[n]]] = torch.nonzero(stay[size[n]:])[:, 0] + size[n]
                src[n, g, :size[n]] = rows.int()
                new_mass[n, g, :size[n]], new_pos[n, g, :size[n]] = m[rows], p[rows]
        dev = s["lens"].device
        src = src.to(dev)
        out = [torch.tensor(size, device=dev, dtype=torch.int32), src, new_mass.to(dev).double(), new_pos.to(dev)]
    page = s["k_cache"].shape[1]
    for x in _caches(s):
        y = x.double()
        for n in range(c["nseq"]):
            for h in range(c["Hkv"]):
                to = src[n, 0 if c["shared"] else h].long()
                to = to[to >= 0]
                at = torch.arange(len(to), device=to.device)
                if s["table"] is None:
                    y[n, at, h] = x[n, to, h].double()
                else:
                    t = s["table"][n].long()
                    y[t[at // page], at % page, h] = x[t[to // page], to % page, h].double()
        out.append(y)
    return out


def _exact_mass(s):
    c = s["case"]
    out = s["mass"].double().clone()
    g, nq, dev = c["Hq"] // c["Hkv"], c["nq"], out.device
    for n in range(c["nseq"]):
        mine = slice(n * nq, (n + 1) * nq)
        length = s["q_len"][mine].long()
        at = torch.arange(int(length.max()), device=dev)
        page = s["k_cache"].shape[1]
        seen = at < length[:, None]
        if s["q_start"] is not None:
            seen = seen & (at >= s["q_start"][mine].long()[:, None])
        for j in range(c["Hq"]):
            k = s["k_cache"][s["table"][n].long()[at // page], at % page, j // g].double()
            x = s["q"][mine, j].double() @ k.t().contiguous() * s["scale"]
            if s["cap"]:
                x = s["cap"] * torch.tanh(x / s["cap"])
            if s["slopes"] is not None:
                x = x - s["slopes"][j].double() * (s["q_pos"][mine].long()[:, None] - at).abs()
            w = torch.exp(x - s["lse"][mine, j].double()[:, None])
            out[n, 0 if c["shared"] else j // g, :len(at)] += torch.where(seen, w, 0.0).sum(0)
    return out


def _exact_sample(s):
    c = s["case"]
    tokens, logs = [], []
    setting = {k: None if s[k] is None else s[k].tolist() for k in ("temperature", "top_k", "top_p", "min_p", "u")}
    for t in range(c["T"]):
        x = s["logits"][t].double()
        temp = setting["temperature"][t]
        if not temp > 0:
            tokens.append(int(torch.nonzero(x == x.max())[0]))
            logs.append(0.0)
            continue
        w = torch.exp((x - x.max()) / temp)
        by = torch.argsort(x, descending=True, stable=True)
        if setting["top_k"] and setting["top_k"][t] > 0:
            by = by[:setting["top_k"][t]]
        if setting["min_p"]:
            by = by[w[by] >= setting["min_p"][t]]
        if setting["top_p"] and setting["top_p"][t] < 1:
            run_ = torch.cumsum(w[by], 0)
            by = by[:max(1, int((run_ < setting["top_p"][t] * run_[-1]).sum()) + 1)]
        ids = by.sort().values
        run_ = torch.cumsum(w[ids], 0)
        i = min(int((run_ <= setting["u"][t] * run_[-1]).sum()), len(ids) - 1)
        tokens.append(int(ids[i]))
        logs.append(math.log(float(w[ids[i]] / run_[-1])))
    dev = s["u"].device
    return torch.tensor(tokens, device=dev, dtype=torch.int32), torch.tensor(logs, device=dev, dtype=torch.float64)
