"""ctypes binding of ``libmisa.so`` (the C ABI declared in include/misa.h).

Argument marshalling only: torch tensors in, device pointers and the current
HIP stream out. Every step of the indexer runs in the library's kernels; there
is no fallback of any kind, and a missing library raises at first use.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmisa.so")

MISA_OK = 0
MISA_ERR_ARG = -1
MISA_ERR_ALIGN = -2
MISA_ERR_WORKSPACE = -3
MISA_ERR_HIP = -4

OP_ROUTE = 1
OP_SCORE_TOPK = 2
OP_HIER_RERANK = 3
OP_DSA_DENSE = 4
OP_INDEXER = 5
OP_HIER_INDEXER = 6
OP_BLOCK_FILTER = 7
OP_BLOCK_INDEXER = 8
OP_PIVOT_INDEXER = 9
OP_ATTEND = 10
OP_ATTEND_SELECTED = 11
OP_ATTEND_SHARED = 12
OP_ATTEND_MASS = 13
OP_CACHE_EVICT = 14

BF16 = 1
FP16 = 2
FP32 = 3

KERNEL_SCORE = 1
KERNEL_TOPK = 2
KERNEL_ROUTE = 3
KERNEL_POOL = 4
KERNEL_GATHER_SCORE = 5

_lib = None

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t

_F32 = ctypes.c_float


class KvCache(ctypes.Structure):
    """misa_kv_cache: where a cache lies and how it is paged."""
    _fields_ = [("k", _P), ("v", _P), ("npages", _I64), ("page", _I64), ("page_stride", _I64), ("token_stride", _I64),
                ("head_stride", _I64), ("heads", _I32), ("d", _I32), ("dtype", _I32), ("table", _P),
                ("table_cols", _I64), ("nseq", _I64)]


_SIGNATURES = {
    "misa_version": (_I32, []),
    "misa_status_string": (ctypes.c_char_p, [_I32]),
    "misa_last_error": (ctypes.c_char_p, []),
    "misa_workspace_bytes": (_SZ, [_I32, _I64, _I32, _I64, _I32, _I32, _I32]),
    "misa_pool_keys": (_I32, [_P, _I64, _I64, _I32, _I32, _P, _P]),
    "misa_pool_update": (_I32, [_P, _I64, _I64, _I32, _I32, _P, _P, _I32, _P, _P]),
    "misa_route": (_I32, [_P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _I64, _I64, _I32, _I32, _P, _P, _P, _SZ, _P]),
    "misa_score_topk": (_I32, [_P, _P, _P, _P, _I32, _P, _P, _I64, _I32, _I32, _I64, _I64, _I32, _P, _P, _P, _SZ,
                               _P]),
    "misa_hier_rerank": (_I32, [_P, _P, _P, _P, _I32, _P, _P, _I64, _I32, _I32, _I64, _I64, _I32, _P, _P, _P, _SZ,
                                _P]),
    "dsa_index_dense": (_I32, [_P, _P, _P, _P, _P, _I64, _I32, _I32, _I64, _I64, _I32, _P, _P, _P, _SZ, _P]),
    "misa_debug_scores": (_I32, [_P, _P, _P, _P, _I32, _P, _P, _I64, _I32, _I32, _I64, _I64, _P, _P]),
    "misa_indexer": (_I32, [_P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _I64, _I64, _I32, _I32, _I32, _P, _P, _P, _P,
                            _SZ, _P]),
    "misa_hier_indexer": (_I32, [_P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _I64, _I64, _I32, _I32, _I32, _I32, _P, _P,
                                 _P, _P, _P, _SZ, _P]),
    "misa_block_filter": (_I32, [_P, _P, _P, _P, _I32, _P, _P, _I64, _I32, _I32, _I64, _I64, _I32, _I32, _P, _P,
                                 _P, _SZ, _P]),
    "misa_block_indexer": (_I32, [_P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _I64, _I64, _I32, _I32, _I32, _I32, _P,
                                  _P, _P, _P, _P, _SZ, _P]),
    "misa_pivot_indexer": (_I32, [_P, _P, _P, _P, _P, _I64, _I32, _I32, _I64, _I64, _I32, _I32, _I32, _P, _P, _P,
                                  _P, _SZ, _P]),
    "misa_hier_indexer_noalloc": (_I32, [_P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _I64, _I64, _I32, _I32, _I32,
                                         _I32, _P, _P, _P, _P, _P]),
    "misa_attend_workspace_bytes": (_SZ, [_I32, _I64, _I32, _I32, _I32, _I64, _I64]),
    "misa_cache_append": (_I32, [_P, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _I32, _P, _P, _P,
                                 _P, _I64, _I32, _I32, _I64, _P]),
    "misa_attend": (_I32, [_P, _P, _I64, _I64, _P, _P, _P, _P, _I64, _I32, _F32, _F32, _P, _P, _P, _P, _SZ, _P]),
    "misa_attend_selected": (_I32, [_P, _P, _I64, _I64, _P, _I32, _P, _P, _P, _I64, _I32, _F32, _F32, _P, _P, _P, _P,
                                    _SZ, _P]),
    "misa_attend_shared": (_I32, [_P, _P, _I64, _I64, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _F32, _F32, _P,
                                  _P, _P, _P, _SZ, _P]),
    "misa_attend_mass": (_I32, [_P, _P, _I64, _I64, _P, _P, _P, _P, _P, _I64, _I32, _F32, _F32, _P, _I32, _P, _P, _P, _SZ,
                                _P]),
    "misa_cache_evict": (_I32, [_P, _P, _P, _P, _I32, _I64, _I64, _I64, _P, _P, _P, _P, _P, _SZ, _P]),
    "misa_cache_move": (_I32, [_P, _P, _I32, _I64, _P]),
    "misa_cache_workspace_bytes": (_SZ, [_I32, _P, _I64, _I32, _I32, _I64]),
    "misa_sample": (_I32, [_P, _I32, _I64, _I64, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "misa_sample_workspace_bytes": (_SZ, [_I64, _I32]),
    "misa_timing_begin": (_I32, [_I32, _I32, _P]),
    "misa_timing_end": (_I32, [_P, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int32)]),
}


class MisaError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} -> {code}: {msg}")
        self.code = code


def lib():
    """Load ``libmisa.so`` (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m routed_token_indexer_amd.build`")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def _check(fn: str, rc: int):
    if rc != MISA_OK:
        raise MisaError(fn, rc, lib().misa_last_error().decode())


def _ptr(x: Optional[torch.Tensor]):
    return None if x is None else ctypes.c_void_p(x.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _req(x: torch.Tensor, dtype, name: str, ndim: int):
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if x.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {x.dtype}")
    if x.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dims, got shape {tuple(x.shape)}")
    if not x.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if not x.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _empty(shape, dtype, device, stream, returned: bool = True, zeros: bool = False):
    """An output or workspace that a call makes itself, from the memory of the stream that it launches on: a block
    that the allocator hands out again then has no user left but earlier work of that stream. What is returned is read
    on the current stream, so its release waits for that one as well."""
    make = torch.zeros if zeros else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        x = make(shape, dtype=dtype, device=device)
    if returned:
        x.record_stream(torch.cuda.current_stream(device))
    return x


def workspace_bytes(op: int, T: int, H: int, Lmax: int, B: int = 0, topk: int = 0, kc: int = 0) -> int:
    return int(lib().misa_workspace_bytes(op, T, H, Lmax, B, topk, kc))


def _workspace(ws: Optional[torch.Tensor], need: int, device, stream) -> torch.Tensor:
    if ws is not None and ws.numel() >= need:
        return ws
    return _empty(max(need, 256), torch.uint8, device, stream, returned=False)


def pool_keys(k: torch.Tensor, B: int, kbar: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Mean of each complete block of B keys: kbar [nseq, Lmax // B, d] fp32."""
    _req(k, torch.bfloat16, "k", 3)
    nseq, L, d = k.shape
    if kbar is None:
        kbar = _empty((nseq, L // B, d), torch.float32, k.device, stream)
    _check("misa_pool_keys", lib().misa_pool_keys(_ptr(k), nseq, L, d, B, _ptr(kbar), _stream(stream)))
    return kbar


def pool_update(k: torch.Tensor, B: int, prev_len: torch.Tensor, new_len: torch.Tensor, max_new: int,
                kbar: torch.Tensor, stream=None) -> torch.Tensor:
    """Pools, in place in ``kbar``, the blocks that growing each sequence from
    ``prev_len`` to ``new_len`` tokens completed (at most ``max_new`` new tokens)."""
    _req(k, torch.bfloat16, "k", 3)
    nseq, L, d = k.shape
    _check("misa_pool_update", lib().misa_pool_update(_ptr(k), nseq, L, d, B, _ptr(prev_len), _ptr(new_len), max_new,
                                                      _ptr(kbar), _stream(stream)))
    return kbar


def route(q, w, k, kbar, q_seq, q_len, B: int, h: int, heads=None, router_key=None, ws=None, stream=None):
    """Routed heads [T, h] (ascending) and, if ``router_key`` is given, the importance r [T, H]."""
    _req(q, torch.bfloat16, "q", 3)
    T, H, d = q.shape
    nseq, L, _ = k.shape
    if heads is None:
        heads = _empty((T, h), torch.int32, q.device, stream)
    ws = _workspace(ws, workspace_bytes(OP_ROUTE, T, H, L, B), q.device, stream)
    _check("misa_route", lib().misa_route(_ptr(q), _ptr(w), _ptr(k), _ptr(kbar), _ptr(q_seq), _ptr(q_len), T, H, d,
                                          nseq, L, B, h, _ptr(heads), _ptr(router_key), _ptr(ws), ws.numel(),
                                          _stream(stream)))
    return heads


def _outs(T, topk, device, idx, score, want_score, stream):
    if idx is None:
        idx = _empty((T, topk), torch.int32, device, stream)
    if score is None and want_score:
        score = _empty((T, topk), torch.float32, device, stream)
    return idx, score


def score_topk(q, w, k, heads, q_seq, q_len, topk: int, idx=None, score=None, want_score=True, ws=None,
               stream=None):
    """Routed scoring + per-query top-k: idx [T, topk] (ascending, -1 padded), score [T, topk]."""
    _req(q, torch.bfloat16, "q", 3)
    _req(heads, torch.int32, "heads", 2)
    T, H, d = q.shape
    nseq, L, _ = k.shape
    idx, score = _outs(T, topk, q.device, idx, score, want_score, stream)
    ws = _workspace(ws, workspace_bytes(OP_SCORE_TOPK, T, H, L, 0, topk), q.device, stream)
    _check("misa_score_topk", lib().misa_score_topk(_ptr(q), _ptr(w), _ptr(k), _ptr(heads), heads.shape[1],
                                                    _ptr(q_seq), _ptr(q_len), T, H, d, nseq, L, topk, _ptr(idx),
                                                    _ptr(score), _ptr(ws), ws.numel(), _stream(stream)))
    return idx, score


def hier_rerank(q, w, k, cand, q_seq, q_len, topk: int, idx=None, score=None, want_score=True, ws=None,
                stream=None):
    """MISA† fine stage: dense re-rank of the candidate rows cand [T, kc] to idx [T, topk]."""
    _req(q, torch.bfloat16, "q", 3)
    _req(cand, torch.int32, "cand", 2)
    T, H, d = q.shape
    nseq, L, _ = k.shape
    kc = cand.shape[1]
    idx, score = _outs(T, topk, q.device, idx, score, want_score, stream)
    ws = _workspace(ws, workspace_bytes(OP_HIER_RERANK, T, H, L, 0, topk, kc), q.device, stream)
    _check("misa_hier_rerank", lib().misa_hier_rerank(_ptr(q), _ptr(w), _ptr(k), _ptr(cand), kc, _ptr(q_seq),
                                                      _ptr(q_len), T, H, d, nseq, L, topk, _ptr(idx), _ptr(score),
                                                      _ptr(ws), ws.numel(), _stream(stream)))
    return idx, score


def dsa_index_dense(q, w, k, q_seq, q_len, topk: int, idx=None, score=None, want_score=True, ws=None,
                    stream=None):
    """Dense DSA indexer (all H heads) + top-k."""
    _req(q, torch.bfloat16, "q", 3)
    T, H, d = q.shape
    nseq, L, _ = k.shape
    idx, score = _outs(T, topk, q.device, idx, score, want_score, stream)
    ws = _workspace(ws, workspace_bytes(OP_DSA_DENSE, T, H, L, 0, topk), q.device, stream)
    _check("dsa_index_dense", lib().dsa_index_dense(_ptr(q), _ptr(w), _ptr(k), _ptr(q_seq), _ptr(q_len), T, H, d,
                                                    nseq, L, topk, _ptr(idx), _ptr(score), _ptr(ws), ws.numel(),
                                                    _stream(stream)))
    return idx, score


def indexer(q, w, k, kbar, q_seq, q_len, B: int, h: int, topk: int, heads=None, idx=None, score=None,
            want_score=True, ws=None, stream=None):
    """Whole MISA indexer (route + routed scoring + top-k) in one call."""
    _req(q, torch.bfloat16, "q", 3)
    T, H, d = q.shape
    nseq, L, _ = k.shape
    idx, score = _outs(T, topk, q.device, idx, score, want_score, stream)
    ws = _workspace(ws, workspace_bytes(OP_INDEXER, T, H, L, B, topk), q.device, stream)
    _check("misa_indexer", lib().misa_indexer(_ptr(q), _ptr(w), _ptr(k), _ptr(kbar), _ptr(q_seq), _ptr(q_len), T, H,
                                              d, nseq, L, B, h, topk, _ptr(heads), _ptr(idx), _ptr(score), _ptr(ws),
                                              ws.numel(), _stream(stream)))
    return idx, score


def hier_indexer(q, w, k, kbar, q_seq, q_len, B: int, h: int, kc: int, topk: int, heads=None, cand=None, idx=None,
                 score=None, want_score=True, ws=None, stream=None):
    """Whole MISA† indexer (route + routed top-k' + dense re-rank to top-k) in one call."""
    _req(q, torch.bfloat16, "q", 3)
    T, H, d = q.shape
    nseq, L, _ = k.shape
    idx, score = _outs(T, topk, q.device, idx, score, want_score, stream)
    ws = _workspace(ws, workspace_bytes(OP_HIER_INDEXER, T, H, L, B, topk, kc), q.device, stream)
    _check("misa_hier_indexer", lib().misa_hier_indexer(_ptr(q), _ptr(w), _ptr(k), _ptr(kbar), _ptr(q_seq),
                                                        _ptr(q_len), T, H, d, nseq, L, B, h, kc, topk, _ptr(heads),
                                                        _ptr(cand), _ptr(idx), _ptr(score), _ptr(ws), ws.numel(),
                                                        _stream(stream)))
    return idx, score


def block_filter(q, w, kbar, heads, q_seq, q_len, Lmax: int, B: int, m: int, blocks=None, cand=None,
                 want_cand=True, ws=None, stream=None):
    """Coarse stage: the m best complete blocks of each query by the routed
    formula on the pooled keys (blocks [T, m], ascending, -1 padded) and the
    candidate token list cand [T, (m + 1) * B] (kept blocks, then the partial one)."""
    _req(q, torch.bfloat16, "q", 3)
    _req(heads, torch.int32, "heads", 2)
    _req(kbar, torch.float32, "kbar", 3)
    T, H, d = q.shape
    nseq = kbar.shape[0]
    if blocks is None:
        blocks = _empty((T, m), torch.int32, q.device, stream)
    if cand is None and want_cand:
        cand = _empty((T, (m + 1) * B), torch.int32, q.device, stream)
    ws = _workspace(ws, workspace_bytes(OP_BLOCK_FILTER, T, H, Lmax, B, 0, m), q.device, stream)
    _check("misa_block_filter", lib().misa_block_filter(_ptr(q), _ptr(w), _ptr(kbar), _ptr(heads), heads.shape[1],
                                                        _ptr(q_seq), _ptr(q_len), T, H, d, nseq, Lmax, B, m,
                                                        _ptr(blocks), _ptr(cand), _ptr(ws), ws.numel(),
                                                        _stream(stream)))
    return blocks, cand


def block_indexer(q, w, k, kbar, q_seq, q_len, B: int, h: int, m: int, topk: int, heads=None, blocks=None, idx=None,
                  score=None, want_score=True, ws=None, stream=None):
    """Route, keep the m best complete blocks (+ the partial one), routed top-k among their tokens."""
    _req(q, torch.bfloat16, "q", 3)
    T, H, d = q.shape
    nseq, L, _ = k.shape
    idx, score = _outs(T, topk, q.device, idx, score, want_score, stream)
    ws = _workspace(ws, workspace_bytes(OP_BLOCK_INDEXER, T, H, L, B, topk, m), q.device, stream)
    _check("misa_block_indexer", lib().misa_block_indexer(_ptr(q), _ptr(w), _ptr(k), _ptr(kbar), _ptr(q_seq),
                                                          _ptr(q_len), T, H, d, nseq, L, B, h, m, topk, _ptr(heads),
                                                          _ptr(blocks), _ptr(idx), _ptr(score), _ptr(ws), ws.numel(),
                                                          _stream(stream)))
    return idx, score


def pivot_indexer(q, w, k, q_seq, q_len, G: int, kc: int, topk: int, cand=None, idx=None, score=None,
                  want_score=True, ws=None, stream=None):
    """PIVOT-Refine over groups of G consecutive queries: the group proxy's dense
    scan keeps kc candidates, each query re-ranks them densely to its top-k."""
    _req(q, torch.bfloat16, "q", 3)
    T, H, d = q.shape
    nseq, L, _ = k.shape
    idx, score = _outs(T, topk, q.device, idx, score, want_score, stream)
    ws = _workspace(ws, workspace_bytes(OP_PIVOT_INDEXER, T, H, L, G, topk, kc), q.device, stream)
    _check("misa_pivot_indexer", lib().misa_pivot_indexer(_ptr(q), _ptr(w), _ptr(k), _ptr(q_seq), _ptr(q_len), T, H,
                                                          d, nseq, L, G, kc, topk, _ptr(cand), _ptr(idx), _ptr(score),
                                                          _ptr(ws), ws.numel(), _stream(stream)))
    return idx, score


def debug_scores(q, w, k, heads, q_seq, q_len, out=None, stream=None):
    """Full routed score rows [T, Lmax] (row t valid for s < q_len[t]); heads=None: dense."""
    _req(q, torch.bfloat16, "q", 3)
    T, H, d = q.shape
    nseq, L, _ = k.shape
    if out is None:
        out = _empty((T, L), torch.float32, q.device, stream, zeros=True)
    h = H if heads is None else heads.shape[1]
    _check("misa_debug_scores", lib().misa_debug_scores(_ptr(q), _ptr(w), _ptr(k), _ptr(heads), h, _ptr(q_seq),
                                                        _ptr(q_len), T, H, d, nseq, L, _ptr(out), _stream(stream)))
    return out


def hier_indexer_noalloc(q, w, k, kbar, q_seq, q_len, B: int, h: int, kc: int, topk: int, heads=None, cand=None,
                         idx=None, score=None, want_score=True, stream=None):
    """misa_hier_indexer with the library's own per-GPU scratch: no workspace,
    nothing allocated by the library (outputs passed in are used as they are)."""
    _req(q, torch.bfloat16, "q", 3)
    T, H, d = q.shape
    nseq, L, _ = k.shape
    idx, score = _outs(T, topk, q.device, idx, score, want_score, stream)
    _check("misa_hier_indexer_noalloc",
           lib().misa_hier_indexer_noalloc(_ptr(q), _ptr(w), _ptr(k), _ptr(kbar), _ptr(q_seq), _ptr(q_len), T, H, d,
                                           nseq, L, B, h, kc, topk, _ptr(heads), _ptr(cand), _ptr(idx), _ptr(score),
                                           _stream(stream)))
    return idx, score


_KV_DTYPES = {torch.bfloat16: BF16, torch.float16: FP16}


def _rows(x: torch.Tensor, name: str, ref: torch.Tensor, n: Optional[int] = None, heads: Optional[int] = None):
    """Token and head strides of a [tokens, heads, d] tensor of ``ref``'s type,
    device and d, rows contiguous."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if x.dtype is not ref.dtype:
        raise TypeError(f"{name}: expected {ref.dtype}, got {x.dtype}")
    if x.device != ref.device:
        raise ValueError(f"{name}: on {x.device}, the cache on {ref.device}")
    shape = x.shape
    if len(shape) != 3 or shape[2] != ref.shape[-1] or (n is not None and shape[0] != n) or \
            (heads is not None and shape[1] != heads):
        raise ValueError(f"{name}: got shape {tuple(shape)}, expected [{'tokens' if n is None else n}, "
                         f"{'heads' if heads is None else heads}, {ref.shape[-1]}]")
    ts, hs, es = x.stride()
    if es != 1 and shape[2] > 1:
        raise ValueError(f"{name}: rows must be contiguous")
    return _stride(shape[0], ts), _stride(shape[1], hs)


def _stride(n: int, s: int) -> int:
    """Stride of an axis of n elements; one of a single element is never used and passes the library's check."""
    return s if n > 1 else 8


def _vec(x: Optional[torch.Tensor], name: str, dtype, shape: tuple, device):
    """Pointer of a contiguous tensor of this dtype and shape (None stays None)."""
    if x is None:
        return None
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if x.dtype is dtype and x.shape == shape and x.device == device and x.is_contiguous():
        return x.data_ptr()
    if x.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {x.dtype}")
    if x.shape != shape:
        raise ValueError(f"{name}: got shape {tuple(x.shape)}, expected {tuple(shape)}")
    if x.device != device:
        raise ValueError(f"{name}: on {x.device}, the cache on {device}")
    raise ValueError(f"{name}: must be contiguous")


def _kv_cache(k_cache: torch.Tensor, v_cache: Optional[torch.Tensor], table: Optional[torch.Tensor]):
    """misa_kv_cache of cache tensors [pages, page, heads, d] (any strides with
    contiguous rows), or [nseq, Lmax, d] for one head without pages."""
    if not isinstance(k_cache, torch.Tensor):
        raise TypeError("k_cache: expected a torch.Tensor")
    dtype = _KV_DTYPES.get(k_cache.dtype)
    if dtype is None:
        raise TypeError(f"k_cache: expected bfloat16 or float16, got {k_cache.dtype}")
    if not k_cache.is_cuda:
        raise ValueError("k_cache: must be a device tensor")
    shape, strides = k_cache.shape, k_cache.stride()
    v = None
    if v_cache is not None:
        if not isinstance(v_cache, torch.Tensor) or v_cache.dtype is not k_cache.dtype:
            raise TypeError(f"v_cache: expected a tensor of {k_cache.dtype}")
        if v_cache.device != k_cache.device:
            raise ValueError(f"v_cache: on {v_cache.device}, k_cache on {k_cache.device}")
        if v_cache.shape != shape or v_cache.stride() != strides:
            raise ValueError("v_cache: must have the shape and strides of k_cache")
        v = v_cache.data_ptr()
    if len(shape) == 4:
        npages, page, heads, d = shape
        ps, ts, hs, es = strides
    elif len(shape) == 3:
        npages, page, d = shape
        heads = 1
        ps, ts, es = strides
        hs = 8
    else:
        raise ValueError(f"k_cache: expected 3 or 4 dims, got shape {tuple(shape)}")
    if es != 1 and d > 1:
        raise ValueError("k_cache: rows must be contiguous")
    nseq, cols, pages = npages, 0, None
    if table is not None:
        if table.dim() != 2:
            raise ValueError(f"table: expected 2 dims, got shape {tuple(table.shape)}")
        nseq, cols = table.shape
        pages = _vec(table, "table", torch.int32, table.shape, k_cache.device)
    return KvCache(k_cache.data_ptr(), v, npages, page, _stride(npages, ps), _stride(page, ts), _stride(heads, hs), heads,
                   d, dtype, pages, cols, nseq)


def _on(device, stream):
    """Stream to launch on: the given one, or the current one of the tensors' device."""
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


_functions = {}


def _call(device, name: str, *args):
    """One library call with ``device`` as the current one."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(lib(), name)
    if torch._C._cuda_getDevice() == device.index:
        rc = fn(*args)
    else:
        with torch.cuda.device(device):
            rc = fn(*args)
    if rc != MISA_OK:
        _check(name, rc)


def attend_workspace_bytes(op: int, T: int, Hq: int, heads: int, d: int, nseq: int, npre: int = 0) -> int:
    return int(lib().misa_attend_workspace_bytes(op, T, Hq, heads, d, nseq, npre))


def cache_append(k, v, k_cache, v_cache, q_seq, q_tok, table=None, q=None, q_out=None, cos_sin=None, pos=None,
                 interleaved=False, stream=None):
    """Append tokens to a cache, rotated on the way; returns ``q_out``.

    k, v [N, heads, d] (v None for a cache of keys alone), q [N, Hq, d] optional;
    k_cache, v_cache [pages, page, heads, d] with ``table`` [nseq, cols] int32, or
    rows of whole sequences ([nseq, Lmax, d] or [nseq, Lmax, heads, d]) without
    one. Token i goes to index ``q_tok[i]`` of sequence ``q_seq[i]`` and is
    rotated by row ``pos[i]`` (default: ``q_tok[i]``) of ``cos_sin`` [P, rot] fp32
    (cosines, then sines; None: no rotation). ``interleaved`` pairs neighbours
    instead of halves. Tokens out of range are skipped.
    """
    c = _kv_cache(k_cache, v_cache, table)
    if (v is None) != (v_cache is None):
        raise ValueError("v and v_cache go together")
    dev = k_cache.device
    k_ts, k_hs = _rows(k, "k", k_cache, None, c.heads)
    N = k.shape[0]
    v_ts, v_hs = (0, 0) if v is None else _rows(v, "v", k_cache, N, c.heads)
    q_ts = q_hs = o_ts = o_hs = Hq = 0
    if q is not None:
        q_ts, q_hs = _rows(q, "q", k_cache, N)
        Hq = q.shape[1]
        if q_out is None:
            q_out = _empty(q.shape, q.dtype, dev, stream)
        o_ts, o_hs = _rows(q_out, "q_out", k_cache, N, Hq)
    elif q_out is not None:
        raise ValueError("q_out without q")
    P = rot = 0
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError(f"cos_sin: expected 2 dims, got shape {tuple(cos_sin.shape)}")
        P, rot = cos_sin.shape
    _call(dev, "misa_cache_append", ctypes.byref(c), k.data_ptr(), k_ts, k_hs, None if v is None else v.data_ptr(), v_ts,
          v_hs, None if q is None else q.data_ptr(), q_ts, q_hs, None if q is None else q_out.data_ptr(), o_ts, o_hs, Hq,
          _vec(q_seq, "q_seq", torch.int32, (N,), dev), _vec(q_tok, "q_tok", torch.int32, (N,), dev),
          _vec(pos, "pos", torch.int32, (N,), dev),
          None if cos_sin is None else _vec(cos_sin, "cos_sin", torch.float32, (P, rot), dev), P, rot, int(interleaved),
          N, _on(dev, stream))
    return q_out


def _attend_common(q, k_cache, v_cache, table, q_seq, q_len, q_pos, scale, slopes, out, lse, want_lse, stream):
    if v_cache is None:
        raise ValueError("v_cache: attention needs values")
    c = _kv_cache(k_cache, v_cache, table)
    dev = k_cache.device
    q_ts, q_hs = _rows(q, "q", k_cache)
    T, Hq, d = q.shape
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _empty((T, Hq, d), q.dtype, dev, stream)
    if lse is None and want_lse:
        lse = _empty((T, Hq), torch.float32, dev, stream)
    ptrs = (_vec(q_seq, "q_seq", torch.int32, (T,), dev), _vec(q_len, "q_len", torch.int32, (T,), dev),
            _vec(q_pos, "q_pos", torch.int32, (T,), dev), _vec(slopes, "slopes", torch.float32, (Hq,), dev),
            _vec(out, "out", k_cache.dtype, (T, Hq, d), dev), _vec(lse, "lse", torch.float32, (T, Hq), dev))
    return c, dev, q_ts, q_hs, T, Hq, float(scale), out, lse, ptrs


def _attend_ws(ws, op, T, Hq, c, dev, stream, npre=0):
    return _scratch(ws, attend_workspace_bytes(op, T, Hq, c.heads, c.d, c.nseq, npre), dev, stream)


def _scratch(ws, need, dev, stream):
    """The given workspace if it is large enough, or one from the stream's memory."""
    if ws is not None:
        if ws.device != dev:
            raise ValueError(f"ws: on {ws.device}, the call on {dev}")
        if ws.dtype is not torch.uint8 or not ws.is_contiguous():
            raise TypeError("ws: expected a contiguous torch.uint8 tensor")
        if ws.numel() >= need:
            return ws
    return _empty(max(need, 256), torch.uint8, dev, stream, returned=False)


def attend(q, k_cache, v_cache, q_seq, q_len, table=None, q_start=None, q_pos=None, scale=None, cap=0.0, slopes=None,
           out=None, lse=None, want_lse=False, ws=None, stream=None):
    """Attention of q [T, Hq, d] over the tokens [q_start, q_len) of their
    sequences' cache (layouts as in ``cache_append``): out [T, Hq, d], lse [T, Hq]
    (natural log; None unless wanted). ``scale`` defaults to d ** -0.5; ``cap``
    > 0 caps the scores by cap * tanh(x / cap); ``slopes`` [Hq] subtracts
    slope * |q_pos - s| (q_pos default: q_len - 1)."""
    c, dev, q_ts, q_hs, T, Hq, scale, out, lse, p = _attend_common(q, k_cache, v_cache, table, q_seq, q_len, q_pos, scale,
                                                                   slopes, out, lse, want_lse, stream)
    ws = _attend_ws(ws, OP_ATTEND, T, Hq, c, dev, stream)
    _call(dev, "misa_attend", ctypes.byref(c), q.data_ptr(), q_ts, q_hs, p[0],
          _vec(q_start, "q_start", torch.int32, (T,), dev), p[1], p[2], T, Hq, scale, cap, p[3], p[4], p[5],
          ws.data_ptr(), ws.numel(), _on(dev, stream))
    return out, lse


def attend_selected(q, k_cache, v_cache, idx, q_seq, q_len, table=None, q_pos=None, scale=None, cap=0.0, slopes=None,
                    out=None, lse=None, want_lse=False, ws=None, stream=None):
    """As ``attend``, over the tokens idx [T, topk] that an indexer selected
    (entries outside [0, q_len) are skipped)."""
    c, dev, q_ts, q_hs, T, Hq, scale, out, lse, p = _attend_common(q, k_cache, v_cache, table, q_seq, q_len, q_pos, scale,
                                                                   slopes, out, lse, want_lse, stream)
    if idx.dim() != 2:
        raise ValueError(f"idx: expected 2 dims, got shape {tuple(idx.shape)}")
    topk = idx.shape[1]
    ws = _attend_ws(ws, OP_ATTEND_SELECTED, T, Hq, c, dev, stream)
    _call(dev, "misa_attend_selected", ctypes.byref(c), q.data_ptr(), q_ts, q_hs,
          _vec(idx, "idx", torch.int32, (T, topk), dev), topk, p[0], p[1], p[2], T, Hq, scale, cap, p[3], p[4], p[5],
          ws.data_ptr(), ws.numel(), _on(dev, stream))
    return out, lse


def attend_shared(q, k_cache, v_cache, q_seq, q_len, pre, pre_len, table=None, pre_table=None, q_pos=None, scale=None,
                  cap=0.0, slopes=None, out=None, lse=None, want_lse=False, ws=None, stream=None):
    """As ``attend``, for sequences that share prefixes: query t sees the
    pre_len[pre[t]] tokens of prefix pre[t] (pages pre_table [npre, cols]; without
    a table prefix i is page i), then the q_len[t] tokens of its own sequence."""
    c, dev, q_ts, q_hs, T, Hq, scale, out, lse, p = _attend_common(q, k_cache, v_cache, table, q_seq, q_len, q_pos, scale,
                                                                   slopes, out, lse, want_lse, stream)
    npre = pre_len.shape[0]
    cols = 0
    if pre_table is not None:
        if pre_table.dim() != 2:
            raise ValueError(f"pre_table: expected 2 dims, got shape {tuple(pre_table.shape)}")
        cols = pre_table.shape[1]
    ws = _attend_ws(ws, OP_ATTEND_SHARED, T, Hq, c, dev, stream, npre)
    _call(dev, "misa_attend_shared", ctypes.byref(c), q.data_ptr(), q_ts, q_hs, p[0], p[1], p[2],
          _vec(pre, "pre", torch.int32, (T,), dev), _vec(pre_len, "pre_len", torch.int32, (npre,), dev),
          None if pre_table is None else _vec(pre_table, "pre_table", torch.int32, (npre, cols), dev), cols, npre, T, Hq,
          scale, cap, p[3], p[4], p[5], ws.data_ptr(), ws.numel(), _on(dev, stream))
    return out, lse


def cache_workspace_bytes(op: int, k_cache, table=None, T: int = 0, Hq: int = 0, lists: int = 1, budget: int = 0) -> int:
    """Workspace bytes of ``attend_mass`` (OP_ATTEND_MASS: T, Hq, lists) or ``cache_evict`` (OP_CACHE_EVICT: lists, budget)."""
    return int(lib().misa_cache_workspace_bytes(op, ctypes.byref(_kv_cache(k_cache, None, table)), T, Hq, lists, budget))


def _cache_ws(ws, op, c, T, Hq, lists, budget, dev, stream):
    return _scratch(ws, int(lib().misa_cache_workspace_bytes(op, ctypes.byref(c), T, Hq, lists, budget)), dev, stream)


def _addressed(c) -> int:
    """Tokens that a sequence of the cache can address."""
    return c.table_cols * c.page if c.table else c.page


def _lists(x, name: str, dtype, c, G, dev):
    """[nseq, lists, tokens] tensor, lists 1 or the cache's heads (G: as another tensor has); its pointer and lists."""
    if x is None:
        return None, G
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if x.dim() != 3 or (x.shape[1] not in (1, c.heads) if G is None else x.shape[1] != G):
        raise ValueError(f"{name}: got shape {tuple(x.shape)}, expected [{c.nseq}, {f'1 or {c.heads}' if G is None else G}, "
                         f"{_addressed(c)}]")
    return _vec(x, name, dtype, (c.nseq, x.shape[1], _addressed(c)), dev), x.shape[1]


def attend_mass(q, k_cache, lse, q_seq, q_len, table=None, q_start=None, q_pos=None, scale=None, cap=0.0, slopes=None,
                mass=None, out=None, per_head=True, ws=None, stream=None):
    """Attention weight that each cached token got, summed over queries and heads.

    Arguments as in ``attend``, whose log-sums ``lse`` [T, Hq] it needs; no values.
    Returns ``out`` [nseq, heads, tokens] fp32 (tokens: as many as a sequence can
    address), or [nseq, 1, tokens] for one sum over all heads, which is what the
    shape of ``mass`` or ``out`` says, or else ``per_head``. ``mass`` is what earlier
    calls gave (None: zeros); ``out`` may be ``mass`` itself.
    """
    c = _kv_cache(k_cache, None, table)
    dev = k_cache.device
    q_ts, q_hs = _rows(q, "q", k_cache)
    T, Hq, d = q.shape
    in_ptr, G = _lists(mass, "mass", torch.float32, c, None, dev)
    out_ptr, G = _lists(out, "out", torch.float32, c, G, dev)
    if G is None:
        G = c.heads if per_head else 1
    if out is None:
        out = _empty((c.nseq, G, _addressed(c)), torch.float32, dev, stream)
        out_ptr = out.data_ptr()
    ptrs = (_vec(lse, "lse", torch.float32, (T, Hq), dev), _vec(q_seq, "q_seq", torch.int32, (T,), dev),
            _vec(q_start, "q_start", torch.int32, (T,), dev), _vec(q_len, "q_len", torch.int32, (T,), dev),
            _vec(q_pos, "q_pos", torch.int32, (T,), dev))
    slopes_ptr = _vec(slopes, "slopes", torch.float32, (Hq,), dev)
    ws = _cache_ws(ws, OP_ATTEND_MASS, c, T, Hq, G, 0, dev, stream)
    _call(dev, "misa_attend_mass", ctypes.byref(c), q.data_ptr(), q_ts, q_hs, *ptrs, T, Hq,
          float(d ** -0.5 if scale is None else scale), cap, slopes_ptr, G, in_ptr, out_ptr, ws.data_ptr(), ws.numel(),
          _on(dev, stream))
    return out


def cache_evict(k_cache, v_cache, mass, lens, budget: int, sinks: int = 0, recent: int = 0, pos=None, table=None,
                mass_out=None, pos_out=None, src=None, new_len=None, ws=None, stream=None):
    """Keeps at most ``budget`` tokens of each sequence and makes them its first rows, in place.

    ``mass`` [nseq, heads, tokens] fp32 (each kv head keeps its own tokens) or
    [nseq, 1, tokens] (all heads the same), ``lens`` [nseq] int32 tokens there are,
    ``pos`` [nseq, lists, tokens] int32 their positions (None: the row numbers). The
    first ``sinks`` positions and the ``recent`` latest ones stay, then the tokens of
    most mass, ties to the lower row. Rows of dropped tokens take the kept rows from
    behind, so rows are in no order afterwards. Returns ``new_len`` [nseq], ``src``
    [nseq, lists, budget] (the row each row came from, -1 behind the last),
    ``mass_out`` and ``pos_out``, where rows have moved along (0 and -1 behind the
    kept ones; they may be ``mass`` and ``pos``). ``new_len`` may be ``lens``,
    ``v_cache`` may be None.
    """
    c = _kv_cache(k_cache, v_cache, table)
    dev = k_cache.device
    if mass is None:
        raise TypeError("mass: expected a torch.Tensor")
    mass_ptr, G = _lists(mass, "mass", torch.float32, c, None, dev)
    pos_ptr, _ = _lists(pos, "pos", torch.int32, c, G, dev)
    if mass_out is None:
        mass_out = _empty(mass.shape, torch.float32, dev, stream)
    if pos_out is None:
        pos_out = _empty(mass.shape, torch.int32, dev, stream)
    if budget < 1:
        raise ValueError(f"budget: {budget} < 1")
    if src is None:
        src = _empty((c.nseq, G, budget), torch.int32, dev, stream)
    if new_len is None:
        new_len = _empty((c.nseq,), torch.int32, dev, stream)
    ws = _cache_ws(ws, OP_CACHE_EVICT, c, 0, 0, G, budget, dev, stream)
    _call(dev, "misa_cache_evict", ctypes.byref(c), mass_ptr, pos_ptr, _vec(lens, "lens", torch.int32, (c.nseq,), dev), G,
          budget, sinks, recent, _lists(mass_out, "mass_out", torch.float32, c, G, dev)[0],
          _lists(pos_out, "pos_out", torch.int32, c, G, dev)[0],
          _vec(src, "src", torch.int32, (c.nseq, G, budget), dev), _vec(new_len, "new_len", torch.int32, (c.nseq,), dev),
          ws.data_ptr(), ws.numel(), _on(dev, stream))
    return new_len, src, mass_out, pos_out


def cache_move(k_cache, v_cache, src, table=None, stream=None):
    """The moves ``src`` [nseq, lists, n] of a ``cache_evict`` in another cache of the same
    sequences, in place: row i takes row src[i] (lists: 1 for all heads, or the cache's
    heads). Entries outside the sequence move nothing."""
    c = _kv_cache(k_cache, v_cache, table)
    dev = k_cache.device
    if not isinstance(src, torch.Tensor):
        raise TypeError("src: expected a torch.Tensor")
    if src.dim() != 3 or src.shape[0] != c.nseq or src.shape[1] not in (1, c.heads):
        raise ValueError(f"src: got shape {tuple(src.shape)}, expected [{c.nseq}, 1 or {c.heads}, rows]")
    _call(dev, "misa_cache_move", ctypes.byref(c), _vec(src, "src", torch.int32, src.shape, dev), src.shape[1],
          src.shape[2], _on(dev, stream))


_LOGIT_DTYPES = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}


def sample_workspace_bytes(T: int, V: int) -> int:
    return int(lib().misa_sample_workspace_bytes(T, V))


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, token=None, logprob=None, want_logprob=False,
           ws=None, stream=None):
    """Next tokens of logits [T, V] (bf16, fp16 or fp32; rows may be strided) from random
    numbers ``u`` [T] in [0, 1): token [T] int32 and its log-probability [T] (None unless wanted).

    Per row, each [T] or None: ``temperature`` (not above 0: the first largest logit),
    then ``top_k`` (not above 0: all), ``min_p`` (of the largest probability), ``top_p``
    (of what the others left). The token is the first one in ascending order whose
    running sum exceeds u times the kept weights' sum; -1 for rows without a finite logit.
    """
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits: expected a torch.Tensor")
    dtype = _LOGIT_DTYPES.get(logits.dtype)
    if dtype is None:
        raise TypeError(f"logits: expected bfloat16, float16 or float32, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError(f"logits: expected 2 dims, got shape {tuple(logits.shape)}")
    if not logits.is_cuda:
        raise ValueError("logits: must be a device tensor")
    dev = logits.device
    T, V = logits.shape
    rs, es = logits.stride()
    if es != 1 and V > 1:
        raise ValueError("logits: rows must be contiguous")
    f32 = torch.float32
    ptrs = [_vec(x, name, dt, (T,), dev) for x, name, dt in
            ((temperature, "temperature", f32), (top_k, "top_k", torch.int32), (top_p, "top_p", f32), (min_p, "min_p", f32))]
    if u is None:
        raise TypeError("u: expected a torch.Tensor")
    u_ptr = _vec(u, "u", f32, (T,), dev)
    if token is None:
        token = _empty((T,), torch.int32, dev, stream)
    if logprob is None and want_logprob:
        logprob = _empty((T,), f32, dev, stream)
    ws = _scratch(ws, sample_workspace_bytes(T, V), dev, stream)
    _call(dev, "misa_sample", logits.data_ptr(), dtype, rs if T > 1 else V, T, V, *ptrs, u_ptr,
          _vec(token, "token", torch.int32, (T,), dev), _vec(logprob, "logprob", f32, (T,), dev), ws.data_ptr(), ws.numel(),
          _on(dev, stream))
    return token, logprob


def timing_begin(kernel: int, capacity: int = 4096, stream=None):
    """Time the launches of one kernel class on ``stream`` (default: the current stream)."""
    _check("misa_timing_begin", lib().misa_timing_begin(kernel, capacity, _stream(stream)))


def timing_end(stream=None):
    ms = ctypes.c_float(0.0)
    n = ctypes.c_int32(0)
    _check("misa_timing_end", lib().misa_timing_end(_stream(stream), ctypes.byref(ms), ctypes.byref(n)))
    return float(ms.value), int(n.value)
