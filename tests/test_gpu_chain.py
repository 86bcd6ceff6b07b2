"""The operators together, as a decode loop uses them: new keys go into the
indexer's cache and the key/value cache, the pooled keys follow, the indexer
selects, and attention reads the selected tokens; then the same tokens by a
whole-prefix attention where everything is selected."""
import pytest
import torch

import attend_oracle as A
from routed_token_indexer_amd import _lib as M

pytestmark = pytest.mark.gpu


def test_decode_loop():
    nseq, Lmax, page, B, H, d, h, topk = 3, 256, 16, 32, 8, 128, 4, 24
    Hq, heads = 16, 2
    bf = torch.bfloat16
    g = torch.Generator().manual_seed(77)
    k_index = torch.zeros(nseq, Lmax, d, dtype=bf, device="cuda")
    kbar = torch.zeros(nseq, Lmax // B, d, device="cuda")
    cols = Lmax // page
    table = torch.randperm(nseq * cols, generator=g).view(nseq, cols).to(torch.int32).cuda()
    kc, vc = (torch.full((nseq * cols, page, heads, d), float("nan"), dtype=bf, device="cuda") for _ in range(2))
    half = 32
    ang = torch.arange(Lmax, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    lens = torch.zeros(nseq, dtype=torch.int32)
    keys = [[] for _ in range(nseq)]                        # what the caches should hold, from the oracle's rotation
    r = lambda *s: torch.randn(*s, generator=g).to(bf).cuda()   # noqa: E731

    def append(seq, tok):
        n = len(seq)
        si, ti = torch.tensor(seq, dtype=torch.int32).cuda(), torch.tensor(tok, dtype=torch.int32).cuda()
        ik, iq, k, v, q = r(n, 1, d), r(n, H, d), r(n, heads, d), r(n, heads, d), r(n, Hq, d)
        iq2 = M.cache_append(ik, None, k_index, None, si, ti, q=iq, cos_sin=cs)
        q2 = M.cache_append(k, v, kc, vc, si, ti, table=table, q=q, cos_sin=cs)
        yk, tk = A.rotate(k.cpu(), cs.cpu(), ti.cpu().long(), False)
        for i in range(n):
            keys[seq[i]].append((yk[i], tk[i], v[i].cpu().double()))
        return si, ti, iq2, q2

    # prompts of uneven length, then single tokens
    prompt = [70, 33, 1]
    seq = [n for n in range(nseq) for _ in range(prompt[n])]
    tok = [t for n in range(nseq) for t in range(prompt[n])]
    prev = lens.clone()
    append(seq, tok)
    lens = torch.tensor(prompt, dtype=torch.int32)
    M.pool_update(k_index, B, prev.cuda(), lens.cuda(), 70, kbar)
    for step in range(12):
        prev = lens.clone()
        si, ti, iq, q = append(list(range(nseq)), lens.tolist())
        lens = lens + 1
        new = lens.cuda()
        M.pool_update(k_index, B, prev.cuda(), new, 1, kbar)
        w = torch.softmax(torch.randn(nseq, H, generator=g), 1).cuda()
        idx, _ = M.indexer(iq.contiguous(), w, k_index, kbar, si, new, B, h, topk)
        out, lse = M.attend_selected(q, kc, vc, idx, si, new, table=table, want_lse=True)
        torch.cuda.synchronize()
        # the pooled keys are those of a full pooling
        full = M.pool_keys(k_index, B)
        for n in range(nseq):
            done = int(lens[n]) // B
            assert torch.equal(kbar[n, :done], full[n, :done])
        A.check((out, lse), A.attend(q, kc, vc, si, new, table=table, idx=idx), f"step {step}")
        if step == 11:
            every = torch.arange(Lmax, dtype=torch.int32, device="cuda").expand(nseq, Lmax).contiguous()
            a = M.attend_selected(q, kc, vc, every, si, new, table=table, want_lse=True)
            b = M.attend(q, kc, vc, si, new, table=table, want_lse=True)
            want = A.attend(q, kc, vc, si, new, table=table)
            A.check(a, want, "everything selected")
            A.check(b, want, "whole prefix")
    for n in range(nseq):
        for s, (k, tol, v) in enumerate(keys[n]):
            p = int(table[n, s // page])
            assert bool(((kc[p, s % page].cpu().double() - k).abs() <= tol).all())
            assert torch.equal(vc[p, s % page].cpu().double(), v)
