"""Python binding of the attention and cache calls (``include/qgemv_attn.h``).

Argument marshalling only, as in the package's ``__init__``; tensors are fp16
or bf16 on the GPU, row offsets and positions int32.  Calls run on the current
stream of the queries' (or the cache's) device and need no synchronization, so
they can be captured in a HIP graph.
"""
from __future__ import annotations

import ctypes
import math

import torch

import gemm_unpack_bit_amd as _q

_DTYPES = {torch.float16: 0, torch.bfloat16: 1}


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token", ctypes.c_int64), ("head", ctypes.c_int64)]


class _Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("layers", "pages", "page_size", "heads_kv", "head_dim", "rows", "max_pages")]
    _fields_ += [(n, ctypes.c_void_p) for n in ("k", "v", "tables", "lens", "refs", "status")]


def _heads(t, name, dtype=None):
    """[tokens, heads, head_dim] view with a contiguous last dimension -> qgemv_heads."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DTYPES or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name} must be {dtype or 'float16 or bfloat16'}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    token, head, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return _Heads(t.data_ptr() or 16, token, head)  # (an empty tensor has no data)


def _ints(t, name, n):
    _q._need(t, torch.int32, name)
    if t.numel() != n:
        raise ValueError(f"{name} must hold {n} int32 values, got {t.numel()}")
    return t.data_ptr()


def _same_device(ref, **others):
    for name, t in others.items():
        if t is not None and t.device != ref.device:
            raise ValueError(f"{name} is on {t.device}, not on {ref.device}")


def _ws(ws, need, device):
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need else None
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous CUDA tensor")
    return ws


def _bytes(ws):
    return (0, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


def attn_prompt_workspace_bytes(tokens, tokens_k, batch, heads, heads_kv, head_dim):
    return int(_q.lib().qgemv_attn_prompt_workspace_bytes(tokens, tokens_k, batch, heads, heads_kv, head_dim))


def attn_tree_workspace_bytes(tokens, rows, heads, heads_kv, head_dim):
    return int(_q.lib().qgemv_attn_tree_workspace_bytes(tokens, rows, heads, heads_kv, head_dim))


def attn_prompt(q, k, v, cu_q, cu_k=None, causal=True, scale=None, out=None, ws=None):
    """Attention over packed prompts: softmax(scale * q k^T) v per sequence.

    q [tokens, heads, head_dim], k and v [tokens_k, heads_kv, head_dim], fp16 or
    bf16, any token and head strides that are multiples of 8 (parts of a fused
    QKV product, say); cu_q, cu_k int32 [batch + 1] row offsets (cu_k None: as
    cu_q).  With ``causal`` the queries of a sequence are its last tokens: query
    i sees keys up to i + nk - nq.  scale: head_dim ** -0.5 by default.  ws:
    optional scratch of attn_prompt_workspace_bytes(...) bytes, reusable across
    calls on one stream.  Returns out [tokens, heads, head_dim]."""
    hq, hk, hv = _heads(q, "q"), _heads(k, "k", q.dtype), _heads(v, "v", q.dtype)
    tokens, heads, dim = q.shape
    tokens_k, heads_kv, _ = k.shape
    if k.shape != v.shape or k.shape[2] != dim:
        raise ValueError("k and v must be [tokens_k, heads_kv, head_dim] with q's head_dim")
    batch = cu_q.numel() - 1
    if batch < 0:
        raise ValueError("cu_q must hold batch + 1 offsets")
    if cu_k is None:
        if tokens_k != tokens:
            raise ValueError("cu_k is needed where queries and keys differ in number")
        cu_k = cu_q
    pq, pk = _ints(cu_q, "cu_q", batch + 1), _ints(cu_k, "cu_k", batch + 1)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    elif out.shape != q.shape:
        raise ValueError("out must have q's shape")
    ho = _heads(out, "out", q.dtype)
    _same_device(q, k=k, v=v, cu_q=cu_q, cu_k=cu_k, out=out, ws=ws)
    if ws is None:
        ws = _ws(None, attn_prompt_workspace_bytes(tokens, tokens_k, batch, heads, heads_kv, dim), q.device)
    else:
        ws = _ws(ws, 0, q.device)
    wp, wn = _bytes(ws)
    _q._check("qgemv_attn_prompt", _q.lib().qgemv_attn_prompt(
        _DTYPES[q.dtype], int(causal), tokens, tokens_k, batch, heads, heads_kv, dim,
        1.0 / math.sqrt(dim) if scale is None else scale, ctypes.byref(hq), ctypes.byref(hk), ctypes.byref(hv), pq, pk,
        ctypes.byref(ho), wp, wn, _q._stream(q)))
    return out


class KvCache:
    """A paged key/value cache: pools k, v [layers, pages, page_size, heads_kv,
    head_dim], and int32 tables [rows, max_pages] (-1: no page), lens [rows],
    refs [pages] (0: free) and status [1] (KV_* bits, set by the calls below and
    cleared by the user).  The tensors are used in place.  ``ws`` is scratch of
    the calls that move pages; calls on one cache and its forks belong on one
    stream, or must be ordered by the caller."""

    def __init__(self, k, v, tables, lens, refs, status=None, ws=None):
        for name, t in (("k", k), ("v", v)):
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise TypeError(f"{name} must be a CUDA tensor")
            if t.dtype not in _DTYPES or t.dtype != k.dtype:
                raise TypeError("k and v must be float16 or bfloat16, and alike")
            if t.dim() != 5 or not t.is_contiguous() or t.shape != k.shape:
                raise ValueError("k and v must be contiguous [layers, pages, page_size, heads_kv, head_dim]")
        if tables.dim() != 2:
            raise ValueError("tables must be [rows, max_pages]")
        rows, max_pages = tables.shape
        if status is None:
            status = torch.zeros(1, dtype=torch.int32, device=k.device)
        for name, t, n in (("tables", tables, rows * max_pages), ("lens", lens, rows), ("refs", refs, k.shape[1]),
                           ("status", status, 1)):
            _ints(t, name, n)
        _same_device(k, v=v, tables=tables, lens=lens, refs=refs, status=status, ws=ws)
        need = int(_q.lib().qgemv_kv_workspace_bytes(rows, k.shape[1]))
        if ws is None:
            ws = torch.empty(max(need, 16), dtype=torch.uint8, device=k.device)
        elif ws.numel() * ws.element_size() < need or not ws.is_contiguous():
            raise ValueError(f"ws must be contiguous and hold {need} bytes")
        self.k, self.v, self.tables, self.lens, self.refs, self.status, self.ws = k, v, tables, lens, refs, status, ws
        self._c = _Cache(*k.shape, rows, max_pages, k.data_ptr(), v.data_ptr(), tables.data_ptr() or 4,
                         lens.data_ptr() or 4, refs.data_ptr(), status.data_ptr())
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, layers, pages, page_size, heads_kv, head_dim, rows, max_pages, dtype=torch.float16, device="cuda"):
        """A cache with no tokens; its pools start as they come."""
        shape = (layers, pages, page_size, heads_kv, head_dim)
        return cls(torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device),
                   torch.full((rows, max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(rows, dtype=torch.int32, device=device),
                   torch.zeros(pages, dtype=torch.int32, device=device))

    def empty_rows(self, rows=None):
        """Another set of (empty) rows over the same pools, for kv_fork's ``out``; as many rows as this one has by
        default."""
        rows = self.rows if rows is None else rows
        return KvCache(self.k, self.v,
                       torch.full((rows, self.max_pages), -1, dtype=torch.int32, device=self.k.device),
                       torch.zeros(rows, dtype=torch.int32, device=self.k.device), self.refs, self.status)

    rows = property(lambda self: self.tables.shape[0])
    max_pages = property(lambda self: self.tables.shape[1])
    page_size = property(lambda self: self.k.shape[2])
    heads_kv = property(lambda self: self.k.shape[3])
    head_dim = property(lambda self: self.k.shape[4])


def kv_reserve(cache, cu, out=None):
    """Grows row b by cu[b + 1] - cu[b] tokens, taking the pages it lacks.
    Returns pos int32 [rows]: where each row's new tokens start, or -1 for a row
    that could not grow (cache.status says why).  Once per step."""
    rows = cache.rows
    pos = torch.empty(rows, dtype=torch.int32, device=cache.k.device) if out is None else out
    p, o = _ints(cu, "cu", rows + 1), _ints(pos, "out", rows)
    _same_device(cache.k, cu=cu, out=pos)
    _q._check("qgemv_kv_reserve", _q.lib().qgemv_kv_reserve(cache._ref, p, o or 4, *_bytes(cache.ws), _q._stream(cache.k)))
    return pos


def kv_write(cache, layer, k, v, cu, pos):
    """Writes one layer's new keys and values [tokens, heads_kv, head_dim] to the
    positions that kv_reserve gave (token cu[b] + i of row b to pos[b] + i)."""
    hk, hv = _heads(k, "k", cache.k.dtype), _heads(v, "v", cache.k.dtype)
    if k.shape != v.shape or tuple(k.shape[1:]) != (cache.heads_kv, cache.head_dim):
        raise ValueError("k and v must be [tokens, heads_kv, head_dim] of the cache")
    p, o = _ints(cu, "cu", cache.rows + 1), _ints(pos, "pos", cache.rows)
    _same_device(cache.k, k=k, v=v, cu=cu, pos=pos)
    _q._check("qgemv_kv_write", _q.lib().qgemv_kv_write(cache._ref, layer, k.shape[0], ctypes.byref(hk), ctypes.byref(hv),
                                                        p, o or 4, _q._stream(cache.k)))


def kv_fork(cache, parents, out=None):
    """Row i of the result is a fork of row parents[i] (int32; -1: an empty row).
    Full pages are shared, a partly filled last page is copied for every child
    but the first, and rows without a child are freed.  ``out`` (by default new
    rows, as many as parents) is a cache over the same pools
    (``cache.empty_rows``) whose tables are overwritten; ``cache``'s own tables
    are stale afterwards.  Returns out."""
    if out is None:
        out = cache.empty_rows(parents.numel())
    p = _ints(parents, "parents", out.rows)
    _same_device(cache.k, parents=parents)
    ws = cache.ws if cache.ws.numel() >= out.ws.numel() else out.ws
    _q._check("qgemv_kv_fork", _q.lib().qgemv_kv_fork(cache._ref, p or 4, out._ref, *_bytes(ws), _q._stream(cache.k)))
    return out


def kv_compact(cache, pos, keep, count):
    """Keeps, of the tokens from position pos[b] on, those at pos[b] +
    keep[b, :count[b]] (ascending), moved together; the rest of the row and the
    pages past its end are given back.  pos, count int32 [rows], keep int32
    [rows, max_keep]; pos -1 leaves a row alone, pos 0 with count 0 frees it."""
    if keep.dim() != 2:
        raise ValueError("keep must be [rows, max_keep]")
    max_keep = keep.shape[1]
    a, b = _ints(pos, "pos", cache.rows), _ints(count, "count", cache.rows)
    c = _ints(keep, "keep", cache.rows * max_keep)
    _same_device(cache.k, pos=pos, keep=keep, count=count)
    _q._check("qgemv_kv_compact", _q.lib().qgemv_kv_compact(cache._ref, a or 4, c or None, max_keep, b or 4,
                                                            *_bytes(cache.ws), _q._stream(cache.k)))


def attn_tree(q, cache, layer, cu, pos, mask=None, scale=None, out=None, ws=None):
    """Attention of new tokens over one layer of a cache.  Row b's tokens
    q[cu[b]:cu[b + 1]] sit at positions pos[b], pos[b] + 1, ... (kv_reserve,
    kv_write); each sees everything before pos[b] and, of the new tokens, those
    in its mask: int64 [tokens, words], bit j of the row's words = token j (a
    drafted tree: its ancestors and itself).  mask None: the new tokens up to
    itself; with one token per row that is a decode step.  ws: optional scratch
    of attn_tree_workspace_bytes(...) bytes.  Returns out, like q."""
    hq = _heads(q, "q", cache.k.dtype)
    tokens, heads, dim = q.shape
    if dim != cache.head_dim:
        raise ValueError("q must have the cache's head_dim")
    words, pm = 0, None
    if mask is not None:
        _q._need(mask, torch.int64, "mask")
        if mask.dim() != 2 or mask.shape[0] != tokens or mask.shape[1] < 1:
            raise ValueError("mask must be [tokens, words]")
        words, pm = mask.shape[1], mask.data_ptr() or 8
    rows = cache.rows
    pc, pp = _ints(cu, "cu", rows + 1), _ints(pos, "pos", rows)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    elif out.shape != q.shape:
        raise ValueError("out must have q's shape")
    ho = _heads(out, "out", q.dtype)
    _same_device(q, cache=cache.k, cu=cu, pos=pos, mask=mask, out=out, ws=ws)
    if ws is None:
        ws = _ws(None, attn_tree_workspace_bytes(tokens, rows, heads, cache.heads_kv, dim), q.device)
    else:
        ws = _ws(ws, 0, q.device)
    wp, wn = _bytes(ws)
    _q._check("qgemv_attn_tree", _q.lib().qgemv_attn_tree(
        _DTYPES[q.dtype], cache._ref, layer, tokens, heads, 1.0 / math.sqrt(dim) if scale is None else scale,
        ctypes.byref(hq), pc, pp or 4, pm, words, ctypes.byref(ho), wp, wn, _q._stream(q)))
    return out
