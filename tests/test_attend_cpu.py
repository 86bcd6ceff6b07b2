"""Host-side checks of the cache and attention calls: every refusal returns
before anything is enqueued (no GPU is needed), workspaces stay bounded, and the
binding checks its tensors."""
import ctypes
import math
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "routed_token_indexer_amd", "libmisa.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmisa.so not built")

FAKE = 1 << 20      # aligned, never dereferenced: validation fails first
ODD = FAKE + 4


@pytest.fixture(scope="module")
def B():
    from routed_token_indexer_amd import _lib
    _lib.lib()
    return _lib


def cache(B, **o):
    c = dict(k=FAKE, v=FAKE, npages=32, page=16, page_stride=16 * 2 * 128, token_stride=2 * 128, head_stride=128, heads=2,
             d=128, dtype=B.BF16, table=FAKE, table_cols=8, nseq=4)
    c.update(o)
    return ctypes.byref(B.KvCache(**c))


BAD_CACHES = [
    (dict(k=None), -1, "key cache"), (dict(dtype=3), -1, "dtype"), (dict(heads=0), -1, "heads"), (dict(npages=0), -1, "npages"),
    (dict(npages=1 << 31), -1, "npages"), (dict(page=0), -1, "page"), (dict(page=1 << 31), -1, "page"),
    (dict(nseq=0), -1, "nseq"), (dict(table_cols=0), -1, "table_cols"), (dict(table_cols=1 << 27), -1, "table_cols"),
    (dict(table=None), -1, "without a table"), (dict(page_stride=0), -2, "strides"), (dict(token_stride=130), -2, "strides"),
    (dict(head_stride=-128), -2, "strides"), (dict(k=ODD), -2, "16-byte"), (dict(v=ODD), -2, "16-byte"),
    (dict(table=FAKE + 1), -2, "table"),
]


def append(B, c, **o):
    a = dict(k=FAKE, k_ts=256, k_hs=128, v=FAKE, v_ts=256, v_hs=128, q=FAKE, q_ts=1024, q_hs=128, q_out=2 * FAKE, o_ts=1024,
             o_hs=128, Hq=8, seq=FAKE, tok=FAKE, pos=None, cs=FAKE, P=100, rot=64, inter=0, N=3)
    a.update(o)
    return B.lib().misa_cache_append(c, *a.values(), None)


def attend(B, c, **o):
    a = dict(q=FAKE, q_ts=1024, q_hs=128, seq=FAKE, start=None, len=FAKE, pos=None, T=3, Hq=8, scale=0.1, cap=0.0,
             slopes=None, out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40)
    a.update(o)
    return B.lib().misa_attend(c, *a.values(), None)


def selected(B, c, **o):
    a = dict(q=FAKE, q_ts=1024, q_hs=128, idx=FAKE, topk=64, seq=FAKE, len=FAKE, pos=None, T=3, Hq=8, scale=0.1, cap=0.0,
             slopes=None, out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40)
    a.update(o)
    return B.lib().misa_attend_selected(c, *a.values(), None)


def shared(B, c, **o):
    a = dict(q=FAKE, q_ts=1024, q_hs=128, seq=FAKE, len=FAKE, pos=None, pre=FAKE, pre_len=FAKE, pre_table=FAKE, pre_cols=4,
             npre=2, T=3, Hq=8, scale=0.1, cap=0.0, slopes=None, out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40)
    a.update(o)
    return B.lib().misa_attend_shared(c, *a.values(), None)


def err(B):
    return B.lib().misa_last_error().decode()


@pytest.mark.parametrize("call", [append, attend, selected, shared])
@pytest.mark.parametrize("bad,code,word", BAD_CACHES)
def test_bad_caches(B, call, bad, code, word):
    assert call(B, cache(B, **bad)) == code
    assert word in err(B)


@pytest.mark.parametrize("call", [append, attend, selected, shared])
def test_null_cache(B, call):
    assert call(B, None) == -1 and "null cache" in err(B)


@pytest.mark.parametrize("bad,code", [
    (dict(N=-1), -1), (dict(Hq=-1), -1), (dict(rot=24), -1), (dict(rot=144), -1), (dict(rot=-16), -1), (dict(P=0), -1),
    (dict(k=None), -1), (dict(v=None), -1), (dict(q=None), -1), (dict(q_out=None), -1), (dict(seq=None), -1),
    (dict(tok=None), -1), (dict(cs=None), -1), (dict(k_ts=100), -2), (dict(k_hs=0), -2), (dict(v_hs=-8), -2),
    (dict(q_ts=1023), -2), (dict(o_hs=4), -2), (dict(k=ODD), -2), (dict(q_out=ODD), -2), (dict(seq=FAKE + 2), -2),
    (dict(q_out=FAKE, o_ts=2048), -1),
])
def test_append_refusals(B, bad, code):
    assert append(B, cache(B), **bad) == code


def test_append_sizes(B):
    assert append(B, cache(B, d=120)) == -1 and "d = 120" in err(B)
    assert append(B, cache(B, d=2048)) == -1
    assert append(B, cache(B, v=None)) == -1 and "go together" in err(B)
    assert append(B, cache(B), N=0) == 0        # nothing to do
    assert append(B, cache(B), N=0, k=None, v=FAKE, q=None, seq=None) == 0


COMMON = [
    (dict(T=-1), -1), (dict(T=1 << 31), -1), (dict(Hq=7), -1), (dict(Hq=0), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1),
    (dict(scale=math.inf), -1), (dict(scale=math.nan), -1), (dict(cap=-1.0), -1), (dict(cap=math.nan), -1),
    (dict(cap=math.inf), -1), (dict(q=None), -1), (dict(seq=None), -1), (dict(len=None), -1), (dict(out=None), -1),
    (dict(q_ts=0), -2), (dict(q_hs=12), -2), (dict(q=ODD), -2), (dict(out=ODD), -2), (dict(lse=FAKE + 2), -2),
    (dict(slopes=FAKE + 2), -2), (dict(pos=FAKE + 1), -2), (dict(ws=None), -3), (dict(ws_bytes=1000), -3),
    (dict(ws=FAKE + 64), -2),
]


@pytest.mark.parametrize("call", [attend, selected, shared])
@pytest.mark.parametrize("bad,code", COMMON)
def test_attention_refusals(B, call, bad, code):
    assert call(B, cache(B), **bad) == code


@pytest.mark.parametrize("call", [attend, selected, shared])
def test_attention_sizes(B, call):
    for d in (32, 96, 512):
        assert call(B, cache(B, d=d)) == -1 and f"d = {d}" in err(B)
    assert call(B, cache(B, v=None)) == -1 and "value cache" in err(B)
    assert call(B, cache(B), T=0) == 0          # nothing to do, no pointer needed
    assert call(B, cache(B), T=0, q=None, seq=None, len=None, out=None, ws=None, ws_bytes=0) == 0


@pytest.mark.parametrize("call", [attend, selected, shared])
def test_grids_and_aliases(B, call):
    """Launches of 2^32 threads or more, and outputs over the queries, are refused as a whole."""
    assert call(B, cache(B), out=2 * FAKE, T=(1 << 31) - 1, Hq=8, ws_bytes=1 << 60) == -1 and "grid" in err(B)
    # one query a workgroup, two kv heads: 2^24 workgroups
    assert selected(B, cache(B), out=2 * FAKE, T=1 << 23) == -1 and "grid" in err(B)
    # four rows a workgroup of the join
    assert shared(B, cache(B), out=2 * FAKE, T=1 << 23, Hq=8, ws_bytes=1 << 60) == -1 and "grid" in err(B)
    assert call(B, cache(B)) == -1 and "must not be q" in err(B)


def test_own_arguments(B):
    assert attend(B, cache(B), start=FAKE + 2) == -2
    assert selected(B, cache(B), topk=0) == -1
    assert selected(B, cache(B), idx=None) == -1
    assert selected(B, cache(B), idx=FAKE + 2) == -2
    assert shared(B, cache(B), npre=0) == -1
    assert shared(B, cache(B), pre=None) == -1
    assert shared(B, cache(B), pre_len=None) == -1
    assert shared(B, cache(B), pre_cols=0) == -1
    assert shared(B, cache(B), pre_len=FAKE + 2) == -2
    assert shared(B, cache(B), pre_table=None, npre=33) == -1 and "npages" in err(B)


def test_workspaces(B):
    w = B.attend_workspace_bytes
    for op in (B.OP_ATTEND, B.OP_ATTEND_SELECTED):
        assert w(op, 0, 64, 8, 128, 4) == 0
        # bounded by the workgroups of a launch, not by the batch or its lengths
        assert 0 < w(op, 4, 64, 8, 128, 4) < 64 << 20
        assert w(op, 100000, 64, 8, 128, 4) < 1 << 20
        assert w(op, 4, 64, 7, 128, 4) == 0 and w(op, 4, 64, 8, 96, 4) == 0
    assert w(B.OP_ATTEND_SHARED, 64, 64, 8, 128, 64, 1) > 64 * 64 * 128 * 4
    assert w(99, 4, 64, 8, 128, 4) == 0


def test_binding_refuses_tensors(B):
    """Types, shapes and devices are checked before the library is called."""
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    kc = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        B.attend(q, kc, kc, i, i)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        B.attend(q, kc.float(), kc.float(), i, i)
    with pytest.raises(ValueError, match="needs values"):
        B.attend(q, kc, None, i, i)
    with pytest.raises(ValueError, match="device tensor"):
        B.cache_append(q[:, :2], q[:, :2], kc, kc, i, i)
    with pytest.raises(ValueError, match="device tensor"):
        B.attend_selected(q, kc, kc, torch.zeros(2, 3, dtype=torch.int32), i, i)
    with pytest.raises(ValueError, match="device tensor"):
        B.attend_shared(q, kc, kc, i, i, i, i)


def test_public_names():
    import routed_token_indexer_amd as misa
    for name in ("cache_append", "attend", "attend_selected", "attend_shared", "attend_workspace_bytes"):
        assert callable(getattr(misa, name))
