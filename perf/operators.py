"""Measured cases of the key/value cache and attention operators.

Four operators, each in a plain form (elementary torch operations in fp32) and
as the library's own call:

  append    rotate new keys (and queries) and store keys and values in a paged cache
  attend    attention over the cache: capped scores, distance bias, visible intervals
  selected  attention over the tokens that an indexer selected
  shared    attention of a batch whose sequences share a long prefix

A query of every attention sees the keys [start, len) of its sequence; a causal
prompt, a decode step, packed documents and a bidirectional prefix differ only
in those two numbers.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token for each of 64 sequences: the append of a decode step, where latency counts
        dict(name="append_decode", op="append", nseq=64, nq=1, L=2048, page=64, Hq=64, Hkv=8, d=128, rot=128,
             pairs="halves", type="bf16", values=True, layout="token"),
        # 4 prompts of 4096 tokens written at once: bound by the bytes moved
        dict(name="append_prompt", op="append", nseq=4, nq=4096, L=4096, page=64, Hq=64, Hkv=8, d=128, rot=128,
             pairs="halves", type="bf16", values=True, layout="token"),
        # the indexer's own key cache (one head, contiguous rows, no values), partial rotation of neighbouring pairs
        dict(name="append_indexer", op="append", nseq=4, nq=1000, L=32768, page=0, Hq=64, Hkv=1, d=128, rot=64,
             pairs="neighbours", type="bf16", values=False, layout="token"),
        # a small decode step of short chats with capped scores
        dict(name="attend_decode_short", op="attend", nseq=8, nq=1, L=1500, page=16, Hq=32, Hkv=8, d=64, mask="causal",
             cap=30.0, bias=False, type="fp16", layout="token"),
        # a decode step over long, uneven prefixes: bound by the cache's bytes
        dict(name="attend_decode_long", op="attend", nseq=8, nq=1, L=32768, page=64, Hq=64, Hkv=8, d=128, mask="causal",
             cap=0.0, bias=False, type="bf16", layout="token"),
        # four positions a step (multi-token decode) with wide heads and a head-major page layout
        dict(name="attend_step_of_4", op="attend", nseq=4, nq=4, L=16384, page=128, Hq=32, Hkv=4, d=256, mask="prefix",
             cap=0.0, bias=True, type="bf16", layout="head"),
        # a causal prompt with capped scores: bound by the matrix cores
        dict(name="attend_prompt_cap", op="attend", nseq=1, nq=8192, L=8192, page=64, Hq=64, Hkv=8, d=128,
             mask="causal", cap=50.0, bias=False, type="bf16", layout="token"),
        # packed documents of uneven length with a distance bias
        dict(name="attend_documents", op="attend", nseq=2, nq=4000, L=4000, page=48, Hq=16, Hkv=4, d=128,
             mask="documents", cap=0.0, bias=True, type="fp16", layout="token"),
        # the tokens that the indexer keeps of four 128K prefixes
        dict(name="selected_decode", op="selected", nseq=4, nq=1, L=131072, page=64, topk=2048, Hq=64, Hkv=1, d=128,
             cap=0.0, type="bf16", layout="token"),
        # the same behind a prompt chunk: every position has a set of its own
        dict(name="selected_prompt", op="selected", nseq=1, nq=2048, L=16384, page=64, topk=2048, Hq=64, Hkv=1, d=128,
             cap=0.0, type="bf16", layout="token"),
        # a small batch behind two system prompts
        dict(name="shared_small", op="shared", npre=2, nseq=6, P=1000, L=100, page=16, Hq=32, Hkv=8, d=64,
             cap=0.0, type="fp16", layout="token"),
        # 64 samples of one 32K prompt
        dict(name="shared_long", op="shared", npre=1, nseq=64, P=32768, L=1000, page=64, Hq=64, Hkv=8, d=128,
             cap=0.0, type="bf16", layout="token"),
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "selected", "shared"])
    Hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, page=rng.choice([1, 16, 24, 48, 64, 128, 256]), Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 3, 4, 7, 8]),
             d=rng.choice([64, 128, 256]), type=rng.choice(["bf16", "fp16"]), layout=rng.choice(["token", "head"]))
    if op == "append":
        N = _log(rng, 1, 12000)
        c["nseq"] = _log(rng, 1, min(N, 200))
        c["nq"] = max(1, N // c["nseq"])
        c["L"] = c["nq"] + _log(rng, 1, 2000)
        c["rot"] = rng.choice([16, 32, 64, c["d"]])
        c["pairs"] = rng.choice(["halves", "neighbours"])
        c["values"] = rng.random() < 0.8
        return c
    c["cap"] = rng.choice([0.0, 0.0, 20.0, 50.0])
    if op == "attend":
        c["mask"] = rng.choice(["causal", "causal", "documents", "prefix"])
        c["bias"] = rng.random() < 0.4
        if rng.random() < 0.6:   # decode and multi-token steps
            c["nseq"], c["nq"] = _log(rng, 1, 48), rng.choice([1, 1, 2, 3, 5])
            c["L"] = _log(rng, max(8, c["nq"]), min(60000, (1 << 28) // (c["nseq"] * c["Hkv"] * c["d"])))
        else:
            c["nseq"] = rng.choice([1, 2, 3])
            c["nq"] = _log(rng, 17, 3000)
            c["L"] = c["nq"] + rng.choice([0, _log(rng, 1, 1000)])
    elif op == "selected":
        c["nseq"], c["nq"] = _log(rng, 1, 16), _log(rng, 1, 64)
        c["topk"] = _log(rng, 1, 2048)
        c["L"] = _log(rng, 16, min(100000, (1 << 28) // (c["nseq"] * c["Hkv"] * c["d"])))
    else:
        c["npre"] = rng.choice([1, 1, 2, 3])
        c["nseq"] = c["npre"] * _log(rng, 1, 24)
        c["P"] = _log(rng, 1, 16000)
        c["L"] = _log(rng, 1, 1500)
    return c


# ---------------------------------------------------------------- lengths (of the case alone)
def _len_of(n, L, least):
    """Uneven lengths of a batch: the first sequence is the longest."""
    return max(least, min(L, int(L * (1.0 - 0.75 * ((n * 0.618034) % 1.0)))))


def _intervals(c):
    """Visible interval [start, len) and position of each query, as three lists."""
    start, length, pos = [], [], []
    for n in range(c["nseq"]):
        total = _len_of(n, c["L"], c.get("nq", 1))
        nq = c.get("nq", 1)
        doc = max(1, total // 7)
        for i in range(nq):
            p = total - nq + i
            a, b = 0, p + 1
            if c.get("mask") == "documents":
                # documents of uneven length: boundaries at multiples of total / 7, every third one left out
                j = p // doc
                a = (j - 1 if j % 3 == 2 else j) * doc
            elif c.get("mask") == "prefix":
                b = max(b, min(total, total // 3))   # the first third sees itself whole
            start.append(a)
            length.append(b)
            pos.append(p)
    return start, length, pos


# ---------------------------------------------------------------- inputs
def _cache(g, c, pages, page, dev, dt):
    """Cache tensor [pages, page, Hkv, d], stored token-major or head-major."""
    Hkv, d = c["Hkv"], c["d"]
    if c["layout"] == "head":
        return torch.randn(pages, Hkv, page, d, generator=g, device=dev, dtype=torch.float32).to(dt).permute(0, 2, 1, 3)
    return torch.randn(pages, page, Hkv, d, generator=g, device=dev, dtype=torch.float32).to(dt)


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt, Hq, Hkv, d = _TYPES[c["type"]], c["Hq"], c["Hkv"], c["d"]
    ints = dict(device=dev, dtype=torch.int32)
    nseq = c["nseq"]
    page = c["page"] or c["L"]
    cols = -(-c["L"] // page)
    s = dict(case=c, scale=1.0 / math.sqrt(d), cap=c.get("cap", 0.0))
    own_pages = nseq * cols
    pre_cols = -(-c["P"] // page) if c["op"] == "shared" else 0
    pages = own_pages + c.get("npre", 0) * pre_cols
    if c["page"]:
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)   # pages lie anywhere in the pool
        s["table"] = order[:own_pages].view(nseq, cols).contiguous()
        s["pre_table"] = order[own_pages:].view(-1, pre_cols).contiguous() if pre_cols else None
    else:
        s["table"] = s["pre_table"] = None
    T = nseq * c.get("nq", 1)
    s["q_seq"] = torch.arange(nseq, **ints).repeat_interleave(c.get("nq", 1))
    if c["op"] == "append":
        fused = torch.randn(T, Hq + 2 * Hkv, d, generator=g, device=dev, dtype=torch.float32).to(dt)
        # q, k and v are slices of one projection's output, as a layer hands them over
        s["q"], s["k"], s["v"] = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:] if c["values"] else None
        s["q_out"] = torch.empty(T, Hq, d, device=dev, dtype=dt)
        s["k_cache"] = _cache(g, c, pages, page, dev, dt)
        s["v_cache"] = _cache(g, c, pages, page, dev, dt) if c["values"] else None
        tok = []
        for n in range(nseq):
            total = _len_of(n, c["L"], c["nq"])
            tok += range(total - c["nq"], total)
        s["q_tok"] = torch.tensor(tok, **ints)
        half = c["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        angle = torch.arange(c["L"], device=dev, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        return s
    s["q"] = (1.5 * torch.randn(T, Hq, d, generator=g, device=dev, dtype=torch.float32)).to(dt)
    s["k_cache"] = _cache(g, c, pages, page, dev, dt)
    s["v_cache"] = _cache(g, c, pages, page, dev, dt)
    start, length, pos = _intervals(c)
    s["q_len"] = torch.tensor(length, **ints)
    s["q_start"] = torch.tensor(start, **ints) if c.get("mask") == "documents" else None
    s["q_pos"] = torch.tensor(pos, **ints) if c.get("bias") else None
    s["slopes"] = (2.0 ** (-8.0 * torch.arange(1, Hq + 1, device=dev, dtype=torch.float32) / Hq)) if c.get("bias") else None
    if c["op"] == "selected":
        # ascending ids without repeats, -1 behind the last one: what the indexer returns. The stride keeps them apart
        k = c["topk"]
        n = torch.clamp(s["q_len"], max=k).long()[:, None]
        j = torch.arange(k, device=dev)[None, :]
        lo, hi = j * s["q_len"][:, None] // n, (j + 1) * s["q_len"][:, None] // n
        u = torch.rand(T, k, generator=g, device=dev)
        ids = lo + (u * (hi - lo)).long().clamp(max=(hi - lo - 1).clamp(min=0))
        s["idx"] = torch.where(j < n, ids, -1).to(torch.int32).contiguous()
    if c["op"] == "shared":
        s["pre"] = (torch.arange(nseq, device=dev) // (nseq // c["npre"])).to(torch.int32)
        s["pre_len"] = torch.tensor([_len_of(i, c["P"], 1) for i in range(c["npre"])], **ints)
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import routed_token_indexer_amd as misa
        if op == "append":
            q = misa.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["q_seq"], s["q_tok"], table=s["table"],
                                  q=s["q"], q_out=s["q_out"], cos_sin=s["cos_sin"],
                                  interleaved=s["case"]["pairs"] == "neighbours")
            return _append_outputs(s, q)
        if op == "attend":
            return misa.attend(s["q"], s["k_cache"], s["v_cache"], s["q_seq"], s["q_len"], table=s["table"],
                               q_start=s["q_start"], q_pos=s["q_pos"], scale=s["scale"], cap=s["cap"],
                               slopes=s["slopes"], want_lse=True)
        if op == "selected":
            return misa.attend_selected(s["q"], s["k_cache"], s["v_cache"], s["idx"], s["q_seq"], s["q_len"],
                                        table=s["table"], scale=s["scale"], cap=s["cap"], want_lse=True)
        return misa.attend_shared(s["q"], s["k_cache"], s["v_cache"], s["q_seq"], s["q_len"], s["pre"], s["pre_len"],
                                  table=s["table"], pre_table=s["pre_table"], scale=s["scale"], cap=s["cap"],
                                  want_lse=True)
    return {"append": _plain_append, "attend": _plain_attend, "selected": _plain_selected, "shared": _plain_shared}[op](s)


def _append_outputs(s, q):
    return [q, s["k_cache"]] if s["v_cache"] is None else [q, s["k_cache"], s["v_cache"]]


def _plain_append(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    row = s["cos_sin"][s["q_tok"].long()]
    cos, sin = row[:, None, :half], row[:, None, half:]

    def rotated(x):
        y = x.float()
        if c["pairs"] == "halves":
            a, b = y[..., :half], y[..., half:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)

    page = s["k_cache"].shape[1]
    seq, tok = s["q_seq"].long(), s["q_tok"].long()
    at = (seq, tok) if s["table"] is None else (s["table"][seq, tok // page].long(), tok % page)
    s["q_out"].copy_(rotated(s["q"]))
    s["k_cache"][at] = rotated(s["k"])
    if s["v_cache"] is not None:
        s["v_cache"][at] = s["v"]
    return _append_outputs(s, s["q_out"])


def _rows(cache, table):
    """The keys (or values) of each sequence in order: fp32 [sequences, Hkv, tokens, d]."""
    x = cache if table is None else cache[table.long()].flatten(1, 2)
    return x.transpose(1, 2).float()


def _heads(q, n, Hkv):
    """Queries of n sequences: fp32 [n, Hkv, queries * heads of one kv head, d]."""
    T, Hq, d = q.shape
    return q.view(n, T // n, Hkv, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(n, Hkv, -1, d).float()


def _capped(x, scale, cap):
    x = x.mul_(scale)
    return x.div_(cap).tanh_().mul_(cap) if cap else x


def _weights(x):
    """exp(x - max) in place of x, its sum and the log of the whole sum; rows of -inf give zeros and -inf."""
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    total = x.sum(-1, keepdim=True)
    return x, total, (m + total.log()).squeeze(-1)


def _plain_attend(s):
    c, Hkv = s["case"], s["case"]["Hkv"]
    nseq, nq, g = c["nseq"], c["nq"], c["Hq"] // Hkv
    x = _capped(_heads(s["q"], nseq, Hkv) @ _rows(s["k_cache"], s["table"]).transpose(-1, -2), s["scale"], s["cap"])
    x = x.view(nseq, Hkv, nq, g, -1)
    at = torch.arange(x.shape[-1], device=x.device)
    per = lambda v: v.view(nseq, 1, nq, 1, 1)  # noqa: E731
    if s["slopes"] is not None:
        x -= s["slopes"].view(1, Hkv, 1, g, 1) * (per(s["q_pos"]) - at).abs()
    hidden = at >= per(s["q_len"])
    if s["q_start"] is not None:
        hidden = hidden | (at < per(s["q_start"]))
    x.masked_fill_(hidden, -math.inf)
    p, total, lse = _weights(x)
    o = p.view(nseq, Hkv, nq * g, -1) @ _rows(s["v_cache"], s["table"])
    o = o.view(nseq, Hkv, nq, g, -1) / total.clamp(min=1e-38)
    return (o.permute(0, 2, 1, 3, 4).reshape(s["q"].shape).to(s["q"].dtype),
            lse.permute(0, 2, 1, 3).reshape(s["q"].shape[:2]))


def _plain_selected(s):
    c, Hkv = s["case"], s["case"]["Hkv"]
    T, Hq, d = s["q"].shape
    page = s["k_cache"].shape[1]
    seen = (s["idx"] >= 0) & (s["idx"] < s["q_len"][:, None])
    ids = torch.where(seen, s["idx"], 0).long()
    pages, slots = s["table"][s["q_seq"].long()[:, None], ids // page].long(), ids % page
    k = s["k_cache"][pages, slots].transpose(1, 2).float()                     # [T, Hkv, topk, d]
    x = _capped(s["q"].view(T, Hkv, Hq // Hkv, d).float() @ k.transpose(-1, -2), s["scale"], s["cap"])
    x.masked_fill_(~seen[:, None, None, :], -math.inf)
    p, total, lse = _weights(x)
    o = p @ s["v_cache"][pages, slots].transpose(1, 2).float() / total.clamp(min=1e-38)
    return o.reshape(T, Hq, d).to(s["q"].dtype), lse.reshape(T, Hq)


def _plain_shared(s):
    c, Hkv = s["case"], s["case"]["Hkv"]
    nseq, npre, g, d = c["nseq"], c["npre"], c["Hq"] // c["Hkv"], c["d"]
    # the prefix's scores for all of its sequences in one product
    a = _heads(s["q"], npre, Hkv) @ _rows(s["k_cache"], s["pre_table"]).transpose(-1, -2)
    a = a.view(npre, Hkv, nseq // npre, g, -1).transpose(1, 2)
    b = (_heads(s["q"], nseq, Hkv) @ _rows(s["k_cache"], s["table"]).transpose(-1, -2)).view(npre, nseq // npre, Hkv, g, -1)
    P, dev = a.shape[-1], a.device
    x = _capped(torch.cat([a, b], -1), s["scale"], s["cap"])
    hidden = torch.cat([(torch.arange(P, device=dev) >= s["pre_len"][:, None]).unsqueeze(1).expand(-1, nseq // npre, -1),
                        (torch.arange(b.shape[-1], device=dev) >= s["q_len"][:, None]).view(npre, nseq // npre, -1)], -1)
    x.masked_fill_(hidden[:, :, None, None, :], -math.inf)
    p, total, lse = _weights(x)
    o = (p[..., :P].transpose(1, 2).reshape(npre, Hkv, -1, P) @ _rows(s["v_cache"], s["pre_table"]))
    o = o.view(npre, Hkv, nseq // npre, g, d).transpose(1, 2).reshape(nseq, Hkv, g, d)
    o = o + p[..., P:].reshape(nseq, Hkv, g, -1) @ _rows(s["v_cache"], s["table"])
    o = o / total.view(nseq, Hkv, g, 1).clamp(min=1e-38)
    return o.reshape(s["q"].shape).to(s["q"].dtype), lse.reshape(s["q"].shape[:2])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    d, Hq, Hkv, T = c["d"], c["Hq"], c["Hkv"], c["nseq"] * c.get("nq", 1)
    if c["op"] == "append":
        heads = Hq + Hkv * (2 if c["values"] else 1)
        positions = len({t for n in range(c["nseq"]) for t in
                         range(_len_of(n, c["L"], c["nq"]) - c["nq"], _len_of(n, c["L"], c["nq"]))})
        return dict(bytes=2 * 2 * T * heads * d + positions * c["rot"] * 4 + 8 * T, flops=3 * T * (Hq + Hkv) * c["rot"])
    row, io = 2 * 2 * Hkv * d, T * Hq * (2 * 2 * d + 4)   # a key with its value; queries, results and their sums
    start, length, _ = _intervals(c)
    if c["op"] == "selected":
        picked = sum(min(c["topk"], n) for n in length)
        # one sequence's queries may share rows: no more than its longest prefix has to be read
        rows = sum(min(max(length[n * c["nq"]:(n + 1) * c["nq"]]),
                       sum(min(c["topk"], x) for x in length[n * c["nq"]:(n + 1) * c["nq"]])) for n in range(c["nseq"]))
        return dict(bytes=rows * row + io + 4 * T * c["topk"], flops=4 * d * Hq * picked)
    if c["op"] == "shared":
        pre = [_len_of(i, c["P"], 1) for i in range(c["npre"])]
        pairs = sum(length) + sum(pre) * (c["nseq"] // c["npre"])
        return dict(bytes=(sum(length) + sum(pre)) * row + io, flops=4 * d * Hq * pairs)
    rows = sum(max(length[n * c["nq"]:(n + 1) * c["nq"]]) - min(start[n * c["nq"]:(n + 1) * c["nq"]]) for n in range(c["nseq"]))
    return dict(bytes=rows * row + io, flops=4 * d * Hq * sum(b - a for a, b in zip(start, length)))


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_rows(scores, scale, cap, bias, seen, v):
    x = scores * scale
    if cap:
        x = cap * torch.tanh(x / cap)
    if bias is not None:
        x = x - bias
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None])
    return p @ v, lse


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "append":
        out = s["q"].double().clone()
        k_cache, v_cache = s["k_cache"].double(), None if s["v_cache"] is None else s["v_cache"].double()
        keys = s["k"].double().clone()
        for i in range(c["rot"] // 2):
            a, b = (i, i + c["rot"] // 2) if c["pairs"] == "halves" else (2 * i, 2 * i + 1)
            co = s["cos_sin"].double()[:, i][s["q_tok"].long()][:, None]
            si = s["cos_sin"].double()[:, i + c["rot"] // 2][s["q_tok"].long()][:, None]
            for x in (out, keys):
                xa, xb = x[:, :, a].clone(), x[:, :, b].clone()
                x[:, :, a], x[:, :, b] = xa * co - xb * si, xb * co + xa * si
        page = k_cache.shape[1]
        for n in range(c["nseq"]):
            mine = slice(n * c["nq"], (n + 1) * c["nq"])
            t = s["q_tok"][mine].long()
            where = torch.full_like(t, n) if s["table"] is None else s["table"][n].long()[t // page]
            k_cache[where, t % page] = keys[mine]
            if v_cache is not None:
                v_cache[where, t % page] = s["v"][mine].double()
        return [out, k_cache] if v_cache is None else [out, k_cache, v_cache]
    T, Hq, d = s["q"].shape
    g, page, dev = Hq // c["Hkv"], s["k_cache"].shape[1], s["q"].device
    o = torch.empty(T, Hq, d, device=dev, dtype=torch.float64)
    lse = torch.empty(T, Hq, device=dev, dtype=torch.float64)
    length = s["q_len"].long()
    first = torch.zeros_like(length) if s.get("q_start") is None else s["q_start"].long()
    nq = c.get("nq", 1)
    if c["op"] == "selected":
        for t in range(0, T, 64):
            t1 = min(T, t + 64)
            ids = s["idx"][t:t1].long()
            seen = (ids >= 0) & (ids < length[t:t1, None])
            ids = ids.clamp(min=0)
            where = torch.gather(s["table"][s["q_seq"][t:t1].long()].long(), 1, ids // page)
            for h in range(c["Hkv"]):
                k, v = (x[where, ids % page, h].double() for x in (s["k_cache"], s["v_cache"]))
                q = s["q"][t:t1, h * g:(h + 1) * g].double()
                o[t:t1, h * g:(h + 1) * g], lse[t:t1, h * g:(h + 1) * g] = _exact_rows(
                    torch.bmm(q, k.transpose(1, 2).contiguous()), s["scale"], s["cap"], None, seen[:, None], v)
        return o, lse
    for n in range(c["nseq"]):
        mine = slice(n * nq, (n + 1) * nq)
        total = int(length[mine].max())
        at = torch.arange(total, device=dev)
        where = s["table"][n].long()[at // page]
        if c["op"] == "shared":
            i = n // (c["nseq"] // c["npre"])
            P = int(s["pre_len"][i])
            ahead = torch.arange(P, device=dev)
        for h in range(c["Hkv"]):
            k, v = (x[where, at % page, h].double() for x in (s["k_cache"], s["v_cache"]))
            seen = (at < length[mine, None]) & (at >= first[mine, None])
            if c["op"] == "shared":
                before = s["pre_table"][i].long()[ahead // page]
                k = torch.cat([s["k_cache"][before, ahead % page, h].double(), k])
                v = torch.cat([s["v_cache"][before, ahead % page, h].double(), v])
                seen = torch.cat([torch.ones(1, P, dtype=torch.bool, device=dev), seen], 1)
            for j in range(h * g, (h + 1) * g):
                bias = s["slopes"][j].double() * (s["q_pos"][mine].long()[:, None] - at).abs() if c.get("bias") else None
                o[mine, j], lse[mine, j] = _exact_rows(s["q"][mine, j].double() @ k.t().contiguous(), s["scale"], s["cap"],
                                                       bias, seen, v)
    return o, lse
