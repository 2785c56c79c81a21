"""Python binding of the norm and sampling calls (``include/qgemv_step.h``).

Argument marshalling only, as in the package's ``__init__``.  Calls run on the
current stream of their tensors' device and need no synchronization, so they
can be captured in a HIP graph.
"""
from __future__ import annotations

import struct

import torch

import gemm_unpack_bit_amd as _q

from .attention import _DTYPES, _done, _kind, _ws

_pack = struct.Struct("Pq").pack  # qgemv_rows: data, row
_lib = _q.lib()
_raw_stream = torch._C._cuda_getCurrentRawStream


def _rows(t, name, shape, dtype, dev):
    """[rows, dim] view with a contiguous last dimension -> a packed qgemv_rows."""
    if t.get_device() != dev or dev < 0:
        raise TypeError(f"{name} must be a CUDA tensor on the same device as the others")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    row, last = t.stride()
    if last != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return _pack(t.data_ptr() or 16, row)  # (an empty tensor has no data)


def _flat(t, name, n, dtype, dev):
    if t.get_device() != dev or dev < 0:
        raise TypeError(f"{name} must be a CUDA tensor on the same device as the others")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must hold {n} contiguous values")
    return t.data_ptr() or 16


def _norm_inputs(x, weight, residual, residual_out):
    dtype, dev, shape = _kind(x, "x"), x.get_device(), x.shape
    if len(shape) != 2:
        raise ValueError("x must be [rows, dim]")
    hx = _rows(x, "x", shape, dtype, dev)
    pw = _flat(weight, "weight", shape[1], dtype, dev)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out goes with residual")
        return dtype, dev, shape, hx, pw, None, None, None
    if residual_out is None:
        residual_out = torch.empty(shape, dtype=dtype, device=x.device)
    return (dtype, dev, shape, hx, pw, _rows(residual, "residual", shape, dtype, dev),
            _rows(residual_out, "residual_out", shape, dtype, dev), residual_out)


def rms_norm(x, weight, eps=1e-6, residual=None, out=None, residual_out=None):
    """y = h * weight / sqrt(mean(h^2) + eps) per row, h = x + residual.

    x, residual [rows, dim], fp16 or bf16, any row strides; weight [dim].
    Returns y, or with a residual (y, h): h rounded once, in ``residual_out``
    (which may be ``residual``, as ``out`` may be ``x``)."""
    dtype, dev, shape, hx, pw, hr, hs, total = _norm_inputs(x, weight, residual, residual_out)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=x.device)
    _done("qgemv_rms_norm", _lib.qgemv_rms_norm(_DTYPES[dtype], *shape, eps, hx, hr, pw, hs,
                                                _rows(out, "out", shape, dtype, dev), _raw_stream(dev)))
    return out if residual is None else (out, total)


def rms_norm_q8(x, weight, eps=1e-6, residual=None, out=None, scales=None, residual_out=None):
    """rms_norm with y in 8 bits for w4a8_rows: int8 codes rint(y / scale) [rows, dim] and fp32 scales [rows], a
    row's max |y| / 127.  Returns (codes, scales), or with a residual (codes, scales, h)."""
    dtype, dev, shape, hx, pw, hr, hs, total = _norm_inputs(x, weight, residual, residual_out)
    rows, dim = shape
    if out is None:
        out = torch.empty(shape, dtype=torch.int8, device=x.device)
    elif out.shape != shape:
        raise ValueError("out must have x's shape")
    if scales is None:
        scales = torch.empty(rows, dtype=torch.float32, device=x.device)
    _done("qgemv_rms_norm_q8", _lib.qgemv_rms_norm_q8(
        _DTYPES[dtype], rows, dim, eps, hx, hr, pw, hs, _flat(out, "out", rows * dim, torch.int8, dev),
        _flat(scales, "scales", rows, torch.float32, dev), _raw_stream(dev)))
    return (out, scales) if residual is None else (out, scales, total)


def w4a8_rows(x8, row_scales, wq, scales, zeros, out=None):
    """The product of w4a8 for activations in 8 bits (rms_norm_q8's): y = (x8 * row_scales) . dequant(Wq)^T, fp16.

    x8 int8 [M, K], M up to 16; row_scales fp32 [M]; wq, scales and zeros as w4a16."""
    dev, shape = x8.get_device(), x8.shape
    if len(shape) != 2:
        raise ValueError("x8 must be [M, K]")
    M, K = shape
    N = scales.shape[0]
    px, pr = _flat(x8, "x8", M * K, torch.int8, dev), _flat(row_scales, "row_scales", M, torch.float32, dev)
    groups = K // _q.GROUP
    need = _lib.qgemv_packed_words(4, _q.LAYOUT_DEVICE, N, K)  # 0 for shapes the library rejects itself
    pq = _flat(wq, "wq", need or wq.numel(), torch.int32, dev)
    ps = _flat(scales, "scales", N * groups, torch.float16, dev)
    pz = _flat(zeros, "zeros", N * -(-groups // 8), torch.int32, dev)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=x8.device)
    elif out.shape != (M, N):
        raise ValueError("out must be [M, N]")
    _done("qgemv_w4a8_rows", _lib.qgemv_w4a8_rows(M, N, K, px, pr, pq, ps, pz, _flat(out, "out", M * N, torch.float16, dev),
                                                  _raw_stream(dev)))
    return out


_LOGITS = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


def sample_workspace_bytes(rows, vocab):
    return int(_lib.qgemv_sample_workspace_bytes(rows, vocab))


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, out=None, ws=None):
    """The next token of every row: int32 [rows].

    logits [rows, vocab], fp16, bf16 or fp32, any row stride; u fp32 [rows]:
    random numbers in [0, 1).  Settings per row, each a tensor [rows] or None:
    temperature fp32 (None: 1; 0: the largest logit), top_k int32 (0: off), top_p
    fp32 (1: off), min_p fp32 (0: off).  Of the tokens by falling logits (equal
    ones by index) the first top_k stay, of those every one with less than top_p
    of their weights in front of it, of those every one with at least min_p of the
    largest's weight; the result is the first token by index up to which the kept
    weights exceed u of their sum (-1: no logit above -infinity).  ws: optional
    scratch of sample_workspace_bytes(rows, vocab) bytes, reusable across calls
    on one stream."""
    if not isinstance(logits, torch.Tensor) or logits.dtype not in _LOGITS:
        raise TypeError("logits must be a float16, bfloat16 or float32 tensor")
    dev = logits.get_device()
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocab]")
    rows, vocab = logits.shape
    if dev < 0:
        raise TypeError("logits must be a CUDA tensor")
    if logits.stride(1) != 1 and vocab > 1:
        raise ValueError("logits must have a contiguous last dimension")
    each = [None if t is None else _flat(t, name, rows, kind, dev) for name, t, kind in (
        ("u", u, torch.float32), ("temperature", temperature, torch.float32), ("top_k", top_k, torch.int32),
        ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32))]
    if out is None:
        out = torch.empty(rows, dtype=torch.int32, device=logits.device)
    if ws is None:
        ws = torch.empty(max(sample_workspace_bytes(rows, vocab), 16), dtype=torch.uint8, device=logits.device)
    wp, wn = _ws(ws, dev)
    _done("qgemv_sample", _lib.qgemv_sample(_LOGITS[logits.dtype], rows, vocab, logits.data_ptr() or 16, logits.stride(0),
                                            *each, _flat(out, "out", rows, torch.int32, dev), wp, wn, _raw_stream(dev)))
    return out
