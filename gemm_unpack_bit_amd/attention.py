"""Python binding of the attention and cache calls (``include/qgemv_attn.h``).

Argument marshalling only, as in the package's ``__init__``; tensors are fp16
or bf16 on the GPU, row offsets and positions int32.  Calls run on the current
stream of the queries' (or the cache's) device and need no synchronization, so
they can be captured in a HIP graph.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

import gemm_unpack_bit_amd as _q

_DTYPES = {torch.float16: 0, torch.bfloat16: 1}
_pack = struct.Struct("Pqq").pack  # qgemv_heads: data, token, head
_lib = _q.lib()
_raw_stream = torch._C._cuda_getCurrentRawStream


class _Cache(ctypes.Structure):  # qgemv_kv_cache
    _fields_ = [(n, ctypes.c_int) for n in ("layers", "pages", "page_size", "heads_kv", "head_dim", "rows", "max_pages")]
    _fields_ += [(n, ctypes.c_void_p) for n in ("k", "v", "tables", "lens", "refs", "status")]


# These checks run on every call of a decode loop, so each is a handful of
# attribute reads; a tensor's device number is -1 off the GPU.

def _heads(t, name, dtype, dev):
    """[tokens, heads, head_dim] view with a contiguous last dimension -> a packed qgemv_heads."""
    if t.get_device() != dev or dev < 0:
        raise TypeError(f"{name} must be a CUDA tensor on the same device as the others")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    stride = t.stride()
    if len(stride) != 3 or stride[2] != 1:
        raise ValueError(f"{name} must be [tokens, heads, head_dim] with a contiguous last dimension")
    return _pack(t.data_ptr() or 16, stride[0], stride[1])  # (an empty tensor has no data)


def _ints(t, name, n, dev):
    if t.get_device() != dev:
        raise TypeError(f"{name} must be a CUDA tensor on the same device as the others")
    if t.dtype is not torch.int32:
        raise TypeError(f"{name} must be {torch.int32}, got {t.dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must hold {n} contiguous int32 values")
    return t.data_ptr() or 4


def _ws(ws, dev):
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous CUDA tensor on the same device as the others")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _kind(t, name):
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be a float16 or bfloat16 tensor")
    return t.dtype


def _done(fn, status):
    if status:
        raise _q.QgemvError(fn, status)


def attn_prompt_workspace_bytes(tokens, tokens_k, batch, heads, heads_kv, head_dim):
    return int(_lib.qgemv_attn_prompt_workspace_bytes(tokens, tokens_k, batch, heads, heads_kv, head_dim))


def attn_tree_workspace_bytes(tokens, rows, heads, heads_kv, head_dim):
    return int(_lib.qgemv_attn_tree_workspace_bytes(tokens, rows, heads, heads_kv, head_dim))


def attn_prompt(q, k, v, cu_q, cu_k=None, causal=True, scale=None, out=None, ws=None):
    """Attention over packed prompts: softmax(scale * q k^T) v per sequence.

    q [tokens, heads, head_dim], k and v [tokens_k, heads_kv, head_dim], fp16 or
    bf16, any token and head strides that are multiples of 8 (parts of a fused
    QKV product, say); cu_q, cu_k int32 [batch + 1] row offsets (cu_k None: as
    cu_q).  With ``causal`` the queries of a sequence are its last tokens: query
    i sees keys up to i + nk - nq.  scale: head_dim ** -0.5 by default.  ws:
    optional scratch of attn_prompt_workspace_bytes(...) bytes, reusable across
    calls on one stream.  Returns out [tokens, heads, head_dim]."""
    dtype, dev = _kind(q, "q"), q.get_device()
    hq, hk, hv = _heads(q, "q", dtype, dev), _heads(k, "k", dtype, dev), _heads(v, "v", dtype, dev)
    tokens, heads, dim = q.shape
    tokens_k, heads_kv, dim_k = k.shape
    if v.shape != k.shape or dim_k != dim:
        raise ValueError("k and v must be [tokens_k, heads_kv, head_dim] with q's head_dim")
    batch = cu_q.numel() - 1
    if batch < 0:
        raise ValueError("cu_q must hold batch + 1 offsets")
    pq = _ints(cu_q, "cu_q", batch + 1, dev)
    if cu_k is not None:
        pk = _ints(cu_k, "cu_k", batch + 1, dev)
    elif tokens_k == tokens:
        pk = pq
    else:
        raise ValueError("cu_k is needed where queries and keys differ in number")
    if out is None:
        out = torch.empty(q.shape, dtype=dtype, device=q.device)
    elif out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if ws is None:
        ws = torch.empty(attn_prompt_workspace_bytes(tokens, tokens_k, batch, heads, heads_kv, dim), dtype=torch.uint8,
                         device=q.device)
    wp, wn = _ws(ws, dev)
    _done("qgemv_attn_prompt", _lib.qgemv_attn_prompt(
        _DTYPES[dtype], int(causal), tokens, tokens_k, batch, heads, heads_kv, dim,
        1.0 / math.sqrt(dim) if scale is None else scale, hq, hk, hv, pq, pk, _heads(out, "out", dtype, dev), wp, wn,
        _raw_stream(dev)))
    return out


class KvCache:
    """A paged key/value cache: pools k, v [layers, pages, page_size, heads_kv,
    head_dim], and int32 tables [rows, max_pages] (-1: no page), lens [rows],
    refs [pages] (0: free) and status [1] (KV_* bits, set by the calls below and
    cleared by the user).  The tensors are used in place.  ``ws`` is scratch of
    the calls that move pages; calls on one cache and its forks belong on one
    stream, or must be ordered by the caller."""

    def __init__(self, k, v, tables, lens, refs, status=None, ws=None):
        dtype, dev = _kind(k, "k"), k.get_device()
        for name, t in (("k", k), ("v", v)):
            if _kind(t, name) is not dtype or t.get_device() != dev or dev < 0:
                raise TypeError("k and v must be CUDA tensors of one type and device")
            if t.dim() != 5 or not t.is_contiguous() or t.shape != k.shape:
                raise ValueError("k and v must be contiguous [layers, pages, page_size, heads_kv, head_dim]")
        if tables.dim() != 2:
            raise ValueError("tables must be [rows, max_pages]")
        rows, max_pages = tables.shape
        if status is None:
            status = torch.zeros(1, dtype=torch.int32, device=k.device)
        pointers = [_ints(t, name, n, dev) for name, t, n in (
            ("tables", tables, rows * max_pages), ("lens", lens, rows), ("refs", refs, k.shape[1]), ("status", status, 1))]
        need = int(_lib.qgemv_kv_workspace_bytes(rows, k.shape[1]))
        if ws is None:
            ws = torch.empty(max(need, 16), dtype=torch.uint8, device=k.device)
        self._ws = _ws(ws, dev)
        if self._ws[1] < need:
            raise ValueError(f"ws must hold {need} bytes")
        self.k, self.v, self.tables, self.lens, self.refs, self.status, self.ws = k, v, tables, lens, refs, status, ws
        self.rows, self.max_pages = rows, max_pages
        self.page_size, self.heads_kv, self.head_dim = k.shape[2:]
        self.dtype, self._dev = dtype, dev
        self._c = _Cache(*k.shape, rows, max_pages, k.data_ptr(), v.data_ptr(), *pointers)
        self._ref = ctypes.addressof(self._c)

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


def kv_reserve(cache, cu, out=None):
    """Grows row b by cu[b + 1] - cu[b] tokens, taking the pages it lacks.
    Returns pos int32 [rows]: where each row's new tokens start, or -1 for a row
    that could not grow (cache.status says why).  Once per step."""
    rows, dev = cache.rows, cache._dev
    if out is None:
        out = torch.empty(rows, dtype=torch.int32, device=cache.k.device)
    _done("qgemv_kv_reserve", _lib.qgemv_kv_reserve(cache._ref, _ints(cu, "cu", rows + 1, dev), _ints(out, "out", rows, dev),
                                                    *cache._ws, _raw_stream(dev)))
    return out


def kv_write(cache, layer, k, v, cu, pos):
    """Writes one layer's new keys and values [tokens, heads_kv, head_dim] to the
    positions that kv_reserve gave (token cu[b] + i of row b to pos[b] + i)."""
    rows, dev, dtype = cache.rows, cache._dev, cache.dtype
    hk, hv = _heads(k, "k", dtype, dev), _heads(v, "v", dtype, dev)
    tokens, heads_kv, dim = k.shape
    if v.shape != k.shape or heads_kv != cache.heads_kv or dim != cache.head_dim:
        raise ValueError("k and v must be [tokens, heads_kv, head_dim] of the cache")
    _done("qgemv_kv_write", _lib.qgemv_kv_write(cache._ref, layer, tokens, hk, hv, _ints(cu, "cu", rows + 1, dev),
                                                _ints(pos, "pos", rows, dev), _raw_stream(dev)))


def kv_fork(cache, parents, out=None):
    """Row i of the result is a fork of row parents[i] (int32; -1: an empty row).
    Full pages are shared, a partly filled last page is copied for every child
    but the first, and rows without a child are freed.  ``out`` (by default new
    rows, as many as parents) is a cache over the same pools
    (``cache.empty_rows``) whose tables are overwritten; ``cache``'s own tables
    are stale afterwards.  Returns out."""
    if out is None:
        out = cache.empty_rows(parents.numel())
    dev = cache._dev
    ws = cache._ws if cache._ws[1] >= out._ws[1] else out._ws
    _done("qgemv_kv_fork", _lib.qgemv_kv_fork(cache._ref, _ints(parents, "parents", out.rows, dev), out._ref, *ws,
                                              _raw_stream(dev)))
    return out


def kv_compact(cache, pos, keep, count):
    """Keeps, of the tokens from position pos[b] on, those at pos[b] +
    keep[b, :count[b]] (ascending), moved together; the rest of the row and the
    pages past its end are given back.  pos, count int32 [rows], keep int32
    [rows, max_keep]; pos -1 leaves a row alone, pos 0 with count 0 frees it."""
    if keep.dim() != 2:
        raise ValueError("keep must be [rows, max_keep]")
    rows, dev, max_keep = cache.rows, cache._dev, keep.shape[1]
    _done("qgemv_kv_compact", _lib.qgemv_kv_compact(
        cache._ref, _ints(pos, "pos", rows, dev), _ints(keep, "keep", rows * max_keep, dev), max_keep,
        _ints(count, "count", rows, dev), *cache._ws, _raw_stream(dev)))


def attn_tree(q, cache, layer, cu, pos, mask=None, scale=None, out=None, ws=None):
    """Attention of new tokens over one layer of a cache.  Row b's tokens
    q[cu[b]:cu[b + 1]] sit at positions pos[b], pos[b] + 1, ... (kv_reserve,
    kv_write); each sees everything before pos[b] and, of the new tokens, those
    in its mask: int64 [tokens, words], bit j of the row's words = token j (a
    drafted tree: its ancestors and itself).  mask None: the new tokens up to
    itself; with one token per row that is a decode step.  ws: optional scratch
    of attn_tree_workspace_bytes(...) bytes.  Returns out, like q."""
    dtype, dev, rows = cache.dtype, cache._dev, cache.rows
    hq = _heads(q, "q", dtype, dev)
    tokens, heads, dim = q.shape
    if dim != cache.head_dim:
        raise ValueError("q must have the cache's head_dim")
    words, pm = 0, None
    if mask is not None:
        if mask.get_device() != dev or mask.dtype is not torch.int64:
            raise TypeError("mask must be an int64 CUDA tensor on the same device as the others")
        if mask.dim() != 2 or mask.shape[0] != tokens or mask.shape[1] < 1 or not mask.is_contiguous():
            raise ValueError("mask must be contiguous [tokens, words]")
        words, pm = mask.shape[1], mask.data_ptr() or 8
    if out is None:
        out = torch.empty(q.shape, dtype=dtype, device=q.device)
    elif out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if ws is None:
        ws = torch.empty(attn_tree_workspace_bytes(tokens, rows, heads, cache.heads_kv, dim), dtype=torch.uint8,
                         device=q.device)
    wp, wn = _ws(ws, dev)
    _done("qgemv_attn_tree", _lib.qgemv_attn_tree(
        _DTYPES[dtype], cache._ref, layer, tokens, heads, 1.0 / math.sqrt(dim) if scale is None else scale, hq,
        _ints(cu, "cu", rows + 1, dev), _ints(pos, "pos", rows, dev), pm, words, _heads(out, "out", dtype, dev), wp, wn,
        _raw_stream(dev)))
    return out
