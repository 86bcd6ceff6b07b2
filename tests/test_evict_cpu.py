"""Host-side checks of accumulated weights, eviction, moves and sampling: every refusal
returns before anything is enqueued, workspaces, what the binding checks, and where a
call on a given stream takes its memory from (no GPU is needed)."""
import ctypes
import math
import os

import pytest
import torch

from test_attend_cpu import B, BAD_CACHES, FAKE, LIB, ODD, cache, err   # noqa: F401  (B is a fixture)
from test_streams_cpu import Stream, check, dev, made                   # noqa: F401  (made is a fixture)

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmisa.so not built")
BYTE = FAKE + 1


def mass(B, c, **o):   # noqa: F811
    a = dict(q=FAKE, q_ts=1024, q_hs=128, lse=FAKE, seq=FAKE, start=None, len=FAKE, pos=None, T=3, Hq=8, scale=0.1, cap=0.0,
             slopes=None, lists=2, inp=None, out=FAKE, ws=FAKE, ws_bytes=1 << 40)
    a.update(o)
    return B.lib().misa_attend_mass(c, *a.values(), None)


def evict(B, c, **o):   # noqa: F811
    a = dict(mass=FAKE, pos=None, lens=FAKE, lists=2, budget=50, sinks=2, recent=10, mass_out=FAKE, pos_out=None, src=FAKE,
             new_len=FAKE, ws=FAKE, ws_bytes=1 << 40)
    a.update(o)
    return B.lib().misa_cache_evict(c, *a.values(), None)


def move(B, c, **o):   # noqa: F811
    a = dict(src=FAKE, lists=1, n=50)
    a.update(o)
    return B.lib().misa_cache_move(c, *a.values(), None)


def sample(B, **o):   # noqa: F811
    a = dict(logits=FAKE, dtype=B.FP32, rs=1000, T=4, V=1000, t=None, k=None, p=None, m=None, u=FAKE, token=FAKE, lp=None,
             ws=FAKE, ws_bytes=1 << 40)
    a.update(o)
    return B.lib().misa_sample(*a.values(), None)


@pytest.mark.parametrize("call", [mass, evict, move])
@pytest.mark.parametrize("bad,code,word", BAD_CACHES)
def test_bad_caches(B, call, bad, code, word):   # noqa: F811
    assert call(B, cache(B, **bad)) == code
    assert word in err(B)


@pytest.mark.parametrize("call", [mass, evict, move])
def test_no_cache_and_lists(B, call):   # noqa: F811
    assert call(B, None) == -1 and "cache" in err(B)
    for lists in (0, -1, 3, 1 << 30):
        assert call(B, cache(B), lists=lists) == -1 and "lists" in err(B)


@pytest.mark.parametrize("o,code,word", [
    (dict(T=-1), -1, "T ="), (dict(T=1 << 31), -1, "T ="), (dict(Hq=0), -1, "Hq"), (dict(Hq=7), -1, "Hq"),
    (dict(Hq=65538), -1, "Hq"), (dict(scale=0.0), -1, "scale"), (dict(scale=math.nan), -1, "scale"), (dict(scale=2e4), -1, "scale"),
    (dict(cap=-1.0), -1, "cap"), (dict(cap=1e-9), -1, "cap"), (dict(cap=math.nan), -1, "cap"), (dict(q=None), -1, "null"),
    (dict(lse=None), -1, "null"), (dict(seq=None), -1, "null"), (dict(len=None), -1, "null"), (dict(out=None), -1, "null"),
    (dict(T=0, out=None), -1, "null"), (dict(q=ODD), -2, "16-byte"), (dict(q_ts=1023), -2, "strides"), (dict(q_hs=0), -2, "strides"),
    (dict(lse=BYTE), -2, "4-byte"), (dict(start=BYTE), -2, "4-byte"), (dict(slopes=BYTE), -2, "4-byte"),
    (dict(inp=BYTE), -2, "4-byte"), (dict(out=BYTE), -2, "4-byte"), (dict(T=1 << 30, Hq=4096), -1, "Hq / heads"),
    (dict(lists=1, ws=None), -3, "workspace"), (dict(lists=1, ws_bytes=16), -3, "workspace"),
    (dict(lists=1, ws=FAKE + 64), -2, "256-byte"),
])
def test_mass_refusals(B, o, code, word):   # noqa: F811
    assert mass(B, cache(B), **o) == code and word in err(B), err(B)


def test_mass_sizes(B):   # noqa: F811
    for d in (32, 96, 512):
        assert mass(B, cache(B, d=d)) == -1 and "d =" in err(B)
    big = dict(page=1 << 20, page_stride=1 << 28, table_cols=1000, nseq=2)
    assert mass(B, cache(B, **big)) == -1 and "grid" in err(B)


@pytest.mark.parametrize("o,code,word", [
    (dict(budget=0), -1, "budget"), (dict(budget=-4), -1, "budget"), (dict(budget=1 << 31), -1, "budget"),
    (dict(sinks=-1), -1, "sinks"), (dict(recent=-1), -1, "recent"), (dict(sinks=51), -1, "sinks"),
    (dict(sinks=41), -1, "sinks"), (dict(sinks=(1 << 63) - 1, recent=(1 << 63) - 1), -1, "sinks"),
    (dict(mass=None), -1, "null"), (dict(lens=None), -1, "null"), (dict(src=None), -1, "null"), (dict(new_len=None), -1, "null"),
    (dict(mass=BYTE), -2, "4-byte"), (dict(pos=BYTE), -2, "4-byte"), (dict(src=BYTE), -2, "4-byte"),
    (dict(mass_out=BYTE), -2, "4-byte"), (dict(ws=None), -3, "workspace"), (dict(ws_bytes=100), -3, "workspace"),
    (dict(ws=FAKE + 128), -2, "256-byte"),
])
def test_evict_refusals(B, o, code, word):   # noqa: F811
    assert evict(B, cache(B), **o) == code and word in err(B), err(B)


@pytest.mark.parametrize("call", [evict, move])
def test_row_sizes(B, call):   # noqa: F811
    for d in (0, 4, 12, 1032):
        assert call(B, cache(B, d=d)) == -1 and "d =" in err(B)
    huge = dict(nseq=1 << 24, table_cols=1)
    assert call(B, cache(B, **huge)) == -1 and "grid" in err(B)


@pytest.mark.parametrize("o,code,word", [(dict(n=-1), -1, "n_src"), (dict(n=1 << 31), -1, "n_src"), (dict(src=None), -1, "null"),
                                         (dict(src=BYTE), -2, "4-byte")])
def test_move_refusals(B, o, code, word):   # noqa: F811
    assert move(B, cache(B), **o) == code and word in err(B), err(B)


def test_nothing_to_move(B):   # noqa: F811
    assert move(B, cache(B), n=0, src=None) == 0


@pytest.mark.parametrize("o,code,word", [
    (dict(dtype=0), -1, "dtype"), (dict(dtype=4), -1, "dtype"), (dict(T=-1), -1, "T ="), (dict(T=1 << 22), -1, "T ="),
    (dict(V=0), -1, "V ="), (dict(V=(1 << 20) + 1), -1, "V ="), (dict(rs=-1), -1, "row_stride"), (dict(rs=1 << 40), -1, "row_stride"),
    (dict(logits=None), -1, "null"), (dict(u=None), -1, "null"), (dict(token=None), -1, "null"), (dict(logits=FAKE + 2), -2, "aligned"),
    (dict(u=BYTE), -2, "4-byte"), (dict(t=BYTE), -2, "4-byte"), (dict(k=BYTE), -2, "4-byte"), (dict(lp=BYTE), -2, "4-byte"),
])
def test_sample_refusals(B, o, code, word):   # noqa: F811
    assert sample(B, **o) == code and word in err(B), err(B)
    assert sample(B, T=0, logits=None, u=None, token=None) == 0


def test_workspaces(B):   # noqa: F811
    size = lambda op, T=0, Hq=0, lists=1, budget=0, **c: B.lib().misa_cache_workspace_bytes(op, cache(B, **c), T, Hq, lists, budget)  # noqa: E731
    # straight to the output: a decode step with a sum per head
    assert size(B.OP_ATTEND_MASS, 4, 8, 2) == 0
    # a sum per head first, then one over the heads: 4 sequences x 2 heads x 128 tokens, fp32
    assert size(B.OP_ATTEND_MASS, 4, 8, 1) == 4 * 2 * 128 * 4
    assert size(B.OP_ATTEND_MASS, 0, 8, 1) == 4 * 2 * 128 * 4
    # a long prompt over few keys: at most 64 parts
    assert 0 < size(B.OP_ATTEND_MASS, 1 << 20, 8, 2) <= 64 * 4 * 2 * 128 * 4
    assert size(B.OP_CACHE_EVICT, lists=2, budget=50) == 3328          # 4 x 2 x 2 x 50 x 4, to 256
    assert size(B.OP_CACHE_EVICT, lists=2, budget=1 << 30) == 4 * 2 * 2 * 128 * 4
    assert size(99, 4, 8, 2) == 0 and size(B.OP_ATTEND_MASS, 4, 7, 2) == 0
    for T, V in ((1, 1), (4, 32000), (64, 128000), (512, 1 << 20)):
        assert B.sample_workspace_bytes(T, V) <= 64 << 20
    assert B.sample_workspace_bytes(0, 1000) == 0


def args():
    bf, i32 = torch.bfloat16, torch.int32
    x = dict(q=torch.randn(2, 4, 64).to(bf), kc=torch.randn(3, 16, 2, 64).to(bf), i=torch.zeros(2, dtype=i32),
             lse=torch.zeros(2, 4), mass=torch.rand(3, 2, 16), lens=torch.zeros(3, dtype=i32),
             src=torch.zeros(3, 2, 5, dtype=i32), logits=torch.randn(2, 9), u=torch.rand(2))
    return {n: dev(t) for n, t in x.items()}


CALLS = {
    "attend_mass": lambda M, x, **o: M.attend_mass(x["q"], x["kc"], x["lse"], x["i"], x["i"], **o),
    "cache_evict": lambda M, x, **o: M.cache_evict(x["kc"], x["kc"], x["mass"], x["lens"], 5, **o),
    "sample": lambda M, x, **o: M.sample(x["logits"], x["u"], want_logprob=True, **o),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_given_streams(made, name):   # noqa: F811
    from routed_token_indexer_amd import _lib as M
    x = args()
    made[0].clear()
    check(made, CALLS[name](M, x, stream=Stream("side")))


@pytest.mark.parametrize("name,change,error", [
    ("attend_mass", dict(lse=torch.zeros(2, 3)), ValueError), ("attend_mass", dict(lse=torch.zeros(2, 4, dtype=torch.float64)), TypeError),
    ("attend_mass", dict(q=torch.randn(2, 4, 64)), TypeError),
    ("attend_mass", dict(q=torch.randn(2, 4, 32).bfloat16()), ValueError), ("attend_mass", dict(i=torch.zeros(3, dtype=torch.int32)), ValueError),
    ("cache_evict", dict(mass=torch.rand(3, 3, 16)), ValueError), ("cache_evict", dict(mass=torch.rand(3, 2, 15)), ValueError),
    ("cache_evict", dict(mass=torch.rand(2, 2, 16)), ValueError), ("cache_evict", dict(mass=torch.rand(3, 2, 16).half()), TypeError),
    ("cache_evict", dict(mass=None), TypeError), ("cache_evict", dict(lens=torch.zeros(3)), TypeError),
    ("sample", dict(logits=torch.randn(2, 9).double()), TypeError), ("sample", dict(logits=torch.randn(9)), ValueError),
    ("sample", dict(logits=torch.randn(9, 2).t()), ValueError), ("sample", dict(u=torch.rand(3)), ValueError),
    ("sample", dict(u=None), TypeError), ("sample", dict(u=torch.rand(2).double()), TypeError),
])
def test_binding_checks(made, name, change, error):   # noqa: F811
    from routed_token_indexer_amd import _lib as M
    x = args()
    x.update({k: None if v is None else dev(v) for k, v in change.items()})
    with pytest.raises(error):
        CALLS[name](M, x)


@pytest.mark.parametrize("change,error", [
    (dict(out=torch.rand(3, 1, 16)), ValueError), (dict(mass=torch.rand(3, 5, 16)), ValueError),
    (dict(q_start=torch.zeros(2)), TypeError), (dict(slopes=torch.zeros(5)), ValueError),
])
def test_mass_options(made, change, error):   # noqa: F811
    from routed_token_indexer_amd import _lib as M
    x = args()
    o = dict(mass=x["mass"])
    o.update({k: dev(v) for k, v in change.items()})
    with pytest.raises(error):
        M.attend_mass(x["q"], x["kc"], x["lse"], x["i"], x["i"], **o)


def test_evict_options(made):   # noqa: F811
    from routed_token_indexer_amd import _lib as M
    x = args()
    for o, error in ((dict(pos=torch.zeros(3, 1, 16, dtype=torch.int32)), ValueError), (dict(pos=torch.zeros(3, 2, 16)), TypeError),
                     (dict(src=torch.zeros(3, 2, 6, dtype=torch.int32)), ValueError), (dict(mass_out=torch.rand(3, 1, 16)), ValueError),
                     (dict(new_len=torch.zeros(2, dtype=torch.int32)), ValueError)):
        with pytest.raises(error):
            M.cache_evict(x["kc"], None, x["mass"], x["lens"], 5, **{k: dev(v) for k, v in o.items()})
    with pytest.raises(ValueError):
        M.cache_evict(x["kc"], None, x["mass"], x["lens"], 0)
    for src, error in ((torch.zeros(2, 2, 5, dtype=torch.int32), ValueError), (torch.zeros(3, 3, 5, dtype=torch.int32), ValueError),
                       (torch.zeros(3, 2, 5), TypeError), (torch.zeros(3, 5, dtype=torch.int32), ValueError)):
        with pytest.raises(error):
            M.cache_move(x["kc"], None, dev(src))


def test_public_names():
    import routed_token_indexer_amd as misa
    for name in ("attend_mass", "cache_evict", "cache_move", "cache_workspace_bytes", "sample", "sample_workspace_bytes"):
        assert callable(getattr(misa, name))
