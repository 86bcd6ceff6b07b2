"""A decode loop with a bounded cache: append, attend, accumulate the weights, sample, evict,
the indexer's keys follow; each step against the oracles, and the loop in a graph."""
import pytest
import torch

import attend_oracle as A
import evict_oracle as O
from routed_token_indexer_amd import _lib as M

pytestmark = pytest.mark.gpu
NSEQ, PAGE, COLS, HQ, HEADS, D, V, BUDGET, SINKS, RECENT = 3, 16, 8, 8, 2, 64, 900, 60, 2, 9
L = PAGE * COLS
BF = torch.bfloat16


class Loop:
    """Caches, weights and positions of some sequences on the device; ``step`` makes one token of each."""

    def __init__(self, lists, seed):
        g = self.g = torch.Generator().manual_seed(seed)
        self.lists = lists
        self.table = torch.randperm(NSEQ * COLS, generator=g).view(NSEQ, COLS).to(torch.int32).cuda()
        self.kc, self.vc = (torch.zeros(NSEQ * COLS, PAGE, HEADS, D, dtype=BF, device="cuda") for _ in range(2))
        self.index = torch.zeros(NSEQ, L, D, dtype=BF, device="cuda")
        half = 16
        ang = torch.arange(400, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        self.cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
        self.head = (torch.randn(HQ * D, V, generator=g) * 0.3).to(BF).cuda()
        self.mass = torch.zeros(NSEQ, lists, L, device="cuda")
        self.pos = torch.full((NSEQ, lists, L), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(NSEQ, dtype=torch.int32, device="cuda")
        self.at = torch.zeros(NSEQ, dtype=torch.int32, device="cuda")      # position of the next token
        self.seq = torch.arange(NSEQ, dtype=torch.int32, device="cuda")

    def tokens(self, n):
        r = lambda *s: torch.randn(*s, generator=self.g).to(BF).cuda()   # noqa: E731
        return r(n, HEADS, D), r(n, HEADS, D), r(n, HQ, D), r(n, 1, D)

    def prompt(self, lens):
        """Prompts, whose last 20 queries' weights are counted."""
        seq = torch.arange(NSEQ, dtype=torch.int32).repeat_interleave(torch.tensor(lens)).cuda()
        tok = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
        k, v, q, ik = self.tokens(len(seq))
        q = M.cache_append(k, v, self.kc, self.vc, seq, tok, table=self.table, q=q, cos_sin=self.cs)
        M.cache_append(ik, None, self.index, None, seq, tok)
        out, lse = M.attend(q, self.kc, self.vc, seq, tok + 1, table=self.table, want_lse=True)
        last = torch.tensor([i for n in range(NSEQ) for i in range(sum(lens[:n]), sum(lens[:n + 1])) if i >= sum(lens[:n + 1]) - 20])
        last = last.cuda()
        args = q[last], self.kc, lse[last], seq[last], tok[last] + 1
        M.attend_mass(*args, table=self.table, out=self.mass)
        O.check_mass(self.mass, O.mass(*args, table=self.table, lists=self.lists), "prompt")
        for n, x in enumerate(lens):
            self.pos[n, :, :x] = torch.arange(x, dtype=torch.int32, device="cuda")
        self.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        self.at.copy_(self.lens)

    def step(self, k, v, q, ik, u, budget):
        """What a program does for one token, and nothing that a graph could not hold."""
        r = {}
        n = self.lens + 1
        M.cache_append(ik, None, self.index, None, self.seq, self.lens)
        q = M.cache_append(k, v, self.kc, self.vc, self.seq, self.lens, table=self.table, q=q, cos_sin=self.cs, pos=self.at)
        self.pos.scatter_(2, self.lens.long()[:, None, None].expand(-1, self.lists, 1),
                          self.at[:, None, None].expand(-1, self.lists, 1))
        out, lse = M.attend(q, self.kc, self.vc, self.seq, n, table=self.table, want_lse=True)
        M.attend_mass(q, self.kc, lse, self.seq, n, table=self.table, mass=self.mass, out=self.mass)
        logits = out.view(NSEQ, -1) @ self.head
        token, logprob = M.sample(logits, u, top_k=self.top_k, top_p=self.top_p, want_logprob=True)
        r.update(q=q, n=n, out=out, lse=lse, mass=self.mass.clone(), pos=self.pos.clone(), logits=logits, token=token,
                 logprob=logprob, kc=self.kc.clone(), vc=self.vc.clone(), index=self.index.clone())
        r["new"], r["src"], _, _ = M.cache_evict(self.kc, self.vc, self.mass, n, budget, sinks=SINKS, recent=RECENT, pos=self.pos,
                                                 table=self.table, mass_out=self.mass, pos_out=self.pos)
        if self.lists == 1:
            M.cache_move(self.index, None, r["src"])
        self.lens.copy_(r["new"])
        self.at += 1
        return r

    def settings(self, top_k, top_p):
        self.top_k = torch.tensor([top_k] * NSEQ, dtype=torch.int32, device="cuda")
        self.top_p = torch.tensor([top_p] * NSEQ, device="cuda")


@pytest.mark.parametrize("lists", [1, HEADS])
def test_decode_loop(lists):
    x = Loop(lists, 31)
    x.settings(50, 0.9)
    x.prompt([100, 41, 59])
    for step in range(14):
        u = torch.rand(NSEQ, generator=x.g)
        before = x.mass.clone()
        r = x.step(*x.tokens(NSEQ), u.cuda(), BUDGET)
        torch.cuda.synchronize()
        where = f"step {step}"
        args = dict(table=x.table)
        A.check((r["out"], r["lse"]), A.attend(r["q"], r["kc"], r["vc"], x.seq, r["n"], **args), where)
        O.check_mass(r["mass"], O.mass(r["q"], r["kc"], r["lse"], x.seq, r["n"], lists=lists, before=before, **args), where)
        for n in range(NSEQ):
            may, _ = O.sample_row(r["logits"][n], float(u[n]), k=50, p=float(x.top_p[n]))
            assert int(r["token"][n]) in may
        new, src, mass, pos = O.evict(r["mass"], r["pos"], r["n"], BUDGET, SINKS, RECENT)
        assert torch.equal(r["new"].cpu(), new) and torch.equal(r["src"].cpu(), src)
        assert torch.equal(x.mass.cpu(), mass) and torch.equal(x.pos.cpu(), pos)
        for now, old in ((x.kc, r["kc"]), (x.vc, r["vc"])):
            assert torch.equal(O.bits(now), O.bits(O.move(old, src, x.table)))
        # the positions that stay: the first ones, the latest ones, nothing twice
        for n in range(NSEQ):
            for h in range(lists):
                held = x.pos[n, h, :int(new[n])].tolist()
                assert len(set(held)) == len(held) and set(range(SINKS)) <= set(held)
                assert set(range(int(x.at[n]) - RECENT, int(x.at[n]))) <= set(held)
        if lists == 1:
            # the indexer over the moved keys: asked for everything it finds every token that stayed
            assert torch.equal(O.bits(x.index), O.bits(O.move(r["index"], src)))
            iq, w = torch.randn(NSEQ, 8, D, generator=x.g).to(BF).cuda(), torch.full((NSEQ, 8), 0.125, device="cuda")
            idx, _ = M.indexer(iq, w, x.index, M.pool_keys(x.index, 16), x.seq, x.lens, 16, 4, BUDGET)
            every = M.attend_selected(r["q"], x.kc, x.vc, idx, x.seq, x.lens, table=x.table, want_lse=True)
            A.check(every, A.attend(r["q"], x.kc, x.vc, x.seq, x.lens, table=x.table), f"selected, {where}")
    assert x.lens.tolist() == [BUDGET, 55, BUDGET]


def test_decode_loop_in_a_graph():
    """One step captured and replayed makes the tokens that the eager loop makes, bit for bit."""
    eager, captured = Loop(HEADS, 32), Loop(HEADS, 32)
    for x in (eager, captured):
        x.settings(0, 0.95)
        x.prompt([64, 30, 90])
    still = [torch.zeros_like(t) for t in eager.tokens(NSEQ)] + [torch.zeros(NSEQ, device="cuda")]
    held = [captured.mass, captured.pos, captured.lens, captured.at, captured.kc, captured.vc, captured.index]
    start = [t.clone() for t in held]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured.step(*still, BUDGET)                 # what libraries set up at their first call
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        r = captured.step(*still, BUDGET)
    for t, old in zip(held, start):
        t.copy_(old)
    for step in range(6):
        new = [*eager.tokens(NSEQ), torch.rand(NSEQ, generator=eager.g).cuda()]
        for t, y in zip(still, new):
            t.copy_(y)
        graph.replay()
        want = eager.step(*new, BUDGET)
        torch.cuda.synchronize()
        for name in ("out", "lse", "mass", "logits", "token", "logprob", "src", "new"):
            assert torch.equal(r[name], want[name]), (step, name)
        for a, b in zip(held, [eager.mass, eager.pos, eager.lens, eager.at, eager.kc, eager.vc, eager.index]):
            assert torch.equal(a, b), step
