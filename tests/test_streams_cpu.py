"""Where a call's own outputs and workspace come from when it is given a stream:
the memory of that stream, so that no queued work of the current one still uses
them, and what is returned is kept for the current stream as well. The library
and the streams are stand-ins here; no GPU is needed."""
import contextlib

import pytest
import torch

from routed_token_indexer_amd import _lib as M


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is a device tensor."""
    is_cuda = property(lambda self: True)


def dev(x):
    return torch.Tensor._make_subclass(OnDevice, x)


class Stream:
    def __init__(self, name):
        self.name = self.cuda_stream = name


@pytest.fixture
def made(monkeypatch):
    """[(tensor, stream it was made under)], {address: streams it was recorded for}, the stream in use at the call."""
    now, log, kept = [Stream("current")], [], {}

    @contextlib.contextmanager
    def under(s):
        now.append(s)
        yield
        now.pop()

    def making(fn):
        def f(*a, **k):
            x = fn(*a, **k)
            log.append((x, now[-1].name))
            return x
        return f

    class Library:
        def __getattr__(self, name):
            return lambda *a: 4096 if name.endswith("workspace_bytes") else 0

    monkeypatch.setattr(M, "lib", lambda: Library())
    monkeypatch.setattr(M, "_call", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(M, "_stream", lambda stream=None: (stream or now[-1]).name)
    monkeypatch.setattr(torch, "empty", making(torch.empty))
    monkeypatch.setattr(torch, "zeros", making(torch.zeros))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda x, s: kept.setdefault(x.data_ptr(), []).append(s.name))
    return log, kept


def check(made, results):
    log, kept = made
    assert log and all(name == "side" for _, name in log), [(tuple(x.shape), name) for x, name in log]
    results = [r for r in (results if isinstance(results, tuple) else (results,)) if r is not None]
    assert results
    for r in results:
        assert "current" in kept.get(r.data_ptr(), []), tuple(r.shape)


def attention():
    bf = torch.bfloat16
    q, kc = dev(torch.randn(2, 4, 64).to(bf)), dev(torch.randn(3, 16, 2, 64).to(bf))
    i = dev(torch.zeros(2, dtype=torch.int32))
    return q, kc, i


@pytest.mark.parametrize("name", ["cache_append", "attend", "attend_selected", "attend_shared"])
def test_cache_and_attention(made, name):
    q, kc, i = attention()
    idx = dev(torch.zeros(2, 5, dtype=torch.int32))
    made[0].clear()
    side = Stream("side")
    if name == "cache_append":
        r = M.cache_append(q[:, :2], q[:, :2], kc, kc, i, i, q=q, stream=side)
    elif name == "attend":
        r = M.attend(q, kc, kc, i, i, want_lse=True, stream=side)
    elif name == "attend_selected":
        r = M.attend_selected(q, kc, kc, idx, i, i, want_lse=True, stream=side)
    else:
        r = M.attend_shared(q, kc, kc, i, i, i, i, want_lse=True, stream=side)
    check(made, r)


INDEXERS = {
    "pool_keys": lambda x, s: M.pool_keys(x["k"], 8, stream=s),
    "route": lambda x, s: M.route(x["q"], x["w"], x["k"], x["kbar"], x["i"], x["i"], 8, 2, stream=s),
    "score_topk": lambda x, s: M.score_topk(x["q"], x["w"], x["k"], x["heads"], x["i"], x["i"], 4, stream=s),
    "hier_rerank": lambda x, s: M.hier_rerank(x["q"], x["w"], x["k"], x["heads"], x["i"], x["i"], 2, stream=s),
    "dsa_index_dense": lambda x, s: M.dsa_index_dense(x["q"], x["w"], x["k"], x["i"], x["i"], 4, stream=s),
    "indexer": lambda x, s: M.indexer(x["q"], x["w"], x["k"], x["kbar"], x["i"], x["i"], 8, 2, 4, stream=s),
    "hier_indexer": lambda x, s: M.hier_indexer(x["q"], x["w"], x["k"], x["kbar"], x["i"], x["i"], 8, 2, 8, 4, stream=s),
    "hier_indexer_noalloc": lambda x, s: M.hier_indexer_noalloc(x["q"], x["w"], x["k"], x["kbar"], x["i"], x["i"], 8, 2, 8,
                                                               4, stream=s),
    "block_filter": lambda x, s: M.block_filter(x["q"], x["w"], x["kbar"], x["heads"], x["i"], x["i"], 32, 8, 2, stream=s),
    "block_indexer": lambda x, s: M.block_indexer(x["q"], x["w"], x["k"], x["kbar"], x["i"], x["i"], 8, 2, 2, 4, stream=s),
    "pivot_indexer": lambda x, s: M.pivot_indexer(x["q"], x["w"], x["k"], x["i"], x["i"], 2, 8, 4, stream=s),
    "debug_scores": lambda x, s: M.debug_scores(x["q"], x["w"], x["k"], None, x["i"], x["i"], stream=s),
}


@pytest.mark.parametrize("name", list(INDEXERS))
def test_indexers(made, name):
    bf, i32 = torch.bfloat16, torch.int32
    x = dict(q=torch.randn(2, 4, 128).to(bf), w=torch.randn(2, 4), k=torch.randn(2, 32, 128).to(bf),
             kbar=torch.randn(2, 4, 128), heads=torch.zeros(2, 2, dtype=i32), i=torch.zeros(2, dtype=i32))
    x = {n: dev(t) for n, t in x.items()}
    made[0].clear()
    check(made, INDEXERS[name](x, Stream("side")))
