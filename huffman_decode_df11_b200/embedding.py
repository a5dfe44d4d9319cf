"""The token embedding on a compressed table: rows by token id
(df11_decode_embedding) and the table's gradient (df11_embedding_gradient).

    >>> d = compress_on_device(table)              # vocab x dim, BF16
    >>> h = decode_embedding(d, ids, scale=dim ** 0.5)
    >>> dw = embedding_gradient(ids, dh, vocab, scale=dim ** 0.5)
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import Df11Device, TensorDesc, _check, _stream_handle, lib
from .linear import _aligned_empty, _on_stream

_TYPES = {torch.bfloat16: 0, torch.float32: 1}
_IDS = {torch.int32: 0, torch.int64: 1}
_MAX_TOKENS = 2 ** 31 - 1


class EmbeddingOp(ctypes.Structure):
    """df11_embedding: the rows to look up and where they go."""
    _fields_ = [("ids", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("out_stride", ctypes.c_uint64), ("rows", ctypes.c_uint32),
                ("dim", ctypes.c_uint32), ("tokens", ctypes.c_uint32),
                ("ids_type", ctypes.c_int32), ("out_type", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class EmbeddingGradOp(ctypes.Structure):
    """df11_embedding_grad: gradients of looked-up rows and where their sums go."""
    _fields_ = [("ids", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("grad_stride", ctypes.c_uint64), ("out_stride", ctypes.c_uint64),
                ("rows", ctypes.c_uint32), ("dim", ctypes.c_uint32), ("tokens", ctypes.c_uint32),
                ("ids_type", ctypes.c_int32), ("grad_type", ctypes.c_int32),
                ("out_type", ctypes.c_int32), ("accumulate", ctypes.c_int32),
                ("scale", ctypes.c_float)]


def _check_ids(ids: torch.Tensor, device) -> torch.Tensor:
    if ids.dtype not in _IDS:
        raise TypeError(f"ids: expected int32 or int64, got {ids.dtype}")
    if ids.device != device:
        raise ValueError(f"ids are on {ids.device}, expected {device}")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    if ids.numel() > _MAX_TOKENS:
        raise ValueError(f"at most {_MAX_TOKENS} tokens per call")
    return ids


def _check_scale(scale) -> float:
    scale = float(scale)
    if not math.isfinite(scale):
        raise ValueError("scale must be finite")
    return scale


def _row_stride(name: str, t: torch.Tensor, tokens: int, dim: int) -> int:
    """Elements between the rows of a tensor of tokens x dim (any leading shape)."""
    if t.numel() == 0 or t.is_contiguous():
        return dim
    if t.dim() != 2 or (dim > 1 and t.stride(1) != 1) or (tokens > 1 and t.stride(0) < dim):
        raise ValueError(f"{name}: contiguous, or two dimensions with contiguous rows")
    return t.stride(0) if tokens > 1 else dim


def _embedding_op(d: Df11Device, ids: torch.Tensor, out: torch.Tensor, scale) -> EmbeddingOp:
    if len(d.shape) != 2 or int(getattr(d, "interleave", 1)) != 1:
        raise ValueError("decode_embedding needs a 2-D table (rows x dim), compressed row-major")
    rows, dim = d.shape
    _check_ids(ids, d.device)
    if out.dtype not in _TYPES:
        raise TypeError(f"out: expected float32 or bfloat16, got {out.dtype}")
    tokens = ids.numel()
    if out.dim() < 1 or out.shape[-1] != dim or out.numel() != tokens * dim:
        raise ValueError(f"out: expected {tokens} rows of {dim}, got {tuple(out.shape)}")
    if out.device != d.device:
        raise ValueError(f"out is on {out.device}, the table on {d.device}")
    return EmbeddingOp(ids.data_ptr(), out.data_ptr(), _row_stride("out", out, tokens, dim), rows,
                       dim, tokens, _IDS[ids.dtype], _TYPES[out.dtype], _check_scale(scale))


def _table_desc(d: Df11Device) -> TensorDesc:
    t = d.desc(torch.empty(0, device=d.device))
    t.out_bf16 = None
    return t


class EmbeddingPlan:
    """A lookup into fixed buffers (a decode loop's token ids and hidden
    states), prepared once: run() is one library call, and reads the ids as they
    are then.  `out` is float32 or BF16, ids.shape + (dim,) or tokens x dim
    with any row stride, on other memory than the ids (refused)."""

    def __init__(self, d: Df11Device, ids: torch.Tensor, out: torch.Tensor, scale: float = 1.0):
        self._op = _embedding_op(d, ids, out, scale)
        self._desc = _table_desc(d)
        self._keep = (d, ids, out)
        self._args = (ctypes.byref(self._desc), ctypes.byref(self._op))
        self._lib = lib()
        self._device = d.device

    @property
    def out(self) -> torch.Tensor:
        return self._keep[2]

    def run(self, err: Optional[torch.Tensor] = None, stream=None):
        if torch.cuda.current_device() != self._device.index:
            with torch.cuda.device(self._device):
                return self.run(err, stream)
        _check(self._lib.df11_decode_embedding(*self._args,
                                               err.data_ptr() if err is not None else None,
                                               _stream_handle(stream)), "df11_decode_embedding")
        return (self._keep[2],)


def decode_embedding(d: Df11Device, ids: torch.Tensor, out: Optional[torch.Tensor] = None,
                     scale: float = 1.0, out_dtype: torch.dtype = torch.bfloat16,
                     err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t] = scale * W[ids[t]] from a compressed table W (rows x dim,
    row-major, as compress and compress_on_device make it), decoding only the
    chunks that hold those rows (df11_decode_embedding).  `ids`: contiguous int32
    or int64, any shape; `out`: float32 or BF16, allocated as ids.shape + (dim,)
    in `out_dtype` if None.  With scale 1 and BF16 the rows come back bit for
    bit.  An id outside the table gives a row of zeros and flags `err`
    (check_device_error).  Asynchronous on `stream` (default: the current
    stream)."""
    with torch.cuda.device(d.device), torch.cuda.stream(_on_stream(stream)):
        if out is None:
            if out_dtype not in _TYPES:
                raise TypeError(f"out_dtype: expected float32 or bfloat16, got {out_dtype}")
            if len(d.shape) != 2:
                raise ValueError("decode_embedding needs a 2-D table (rows x dim)")
            out = torch.empty(*ids.shape, d.shape[1], dtype=out_dtype, device=d.device)
        return EmbeddingPlan(d, ids, out, scale).run(err, stream)[0]


def embedding_gradient(ids: torch.Tensor, grad: torch.Tensor, rows: int,
                       out: Optional[torch.Tensor] = None, scale: float = 1.0,
                       accumulate: bool = False, out_dtype: torch.dtype = torch.float32,
                       err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient of decode_embedding's table (rows x dim): dW[v] = scale * the
    sum of grad[t] over the tokens t with ids[t] = v (df11_embedding_gradient).
    `grad`: float32 or BF16, ids.shape + (dim,), or tokens x dim with any row
    stride.  `out`: float32 or BF16, rows x dim with any row stride, allocated in
    `out_dtype` if None.  With `accumulate` the sums are added to `out`, and rows
    without a token are not touched; otherwise those are set to zero.  `out` may not
    share memory with `grad` or `ids` (refused).  Sums run in
    fp32 in token order within pieces of the sorted list: the same call gives
    the same bits.  An id outside the table adds nothing and flags `err`.
    Asynchronous on `stream` (default: the current stream)."""
    rows = int(rows)
    if grad.dtype not in _TYPES:
        raise TypeError(f"grad: expected float32 or bfloat16, got {grad.dtype}")
    if not grad.is_cuda:
        raise ValueError("embedding_gradient takes CUDA tensors")
    _check_ids(ids, grad.device)
    tokens = ids.numel()
    if grad.dim() < 1 or grad.shape[-1] == 0:
        raise ValueError("grad: expected rows of dim elements")
    dim = grad.shape[-1]
    if grad.numel() != tokens * dim:
        raise ValueError(f"grad: expected {tokens} rows of {dim}, got {tuple(grad.shape)}")
    if not 0 < rows < 2 ** 31:
        raise ValueError("rows must be positive and below 2^31")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if stream is not None or torch.cuda.current_device() != grad.device.index:
        # the output and the workspace are allocated (and freed) in the order of the call's stream
        with torch.cuda.device(grad.device), torch.cuda.stream(_on_stream(stream)):
            return _embedding_gradient(ids, grad, rows, out, scale, accumulate, out_dtype, err)
    return _embedding_gradient(ids, grad, rows, out, scale, accumulate, out_dtype, err)


def _embedding_gradient(ids, grad, rows, out, scale, accumulate, out_dtype, err):
    tokens, dim, dev = ids.numel(), grad.shape[-1], grad.device
    if out is None:
        if out_dtype not in _TYPES:
            raise TypeError(f"out_dtype: expected float32 or bfloat16, got {out_dtype}")
        out = torch.empty((rows, dim), dtype=out_dtype, device=dev)
    elif out.dtype not in _TYPES:
        raise TypeError(f"out: expected float32 or bfloat16, got {out.dtype}")
    elif out.shape != (rows, dim) or out.device != dev:
        raise ValueError(f"out: expected {rows} x {dim} on {dev}, got {tuple(out.shape)} on "
                         f"{out.device}")
    op = EmbeddingGradOp(ids.data_ptr(), grad.data_ptr(), out.data_ptr(),
                         _row_stride("grad", grad, tokens, dim), _row_stride("out", out, rows, dim),
                         rows, dim, tokens, _IDS[ids.dtype], _TYPES[grad.dtype], _TYPES[out.dtype],
                         1 if accumulate else 0, _check_scale(scale))
    L, size, ref = lib(), ctypes.c_size_t(0), ctypes.byref(op)
    _check(L.df11_embedding_gradient_workspace(ref, ctypes.byref(size)),
           "df11_embedding_gradient_workspace")
    work = _aligned_empty(size.value, dev)
    _check(L.df11_embedding_gradient(ref, work.data_ptr(), size.value,
                                     err.data_ptr() if err is not None else None,
                                     _stream_handle(None)),
           "df11_embedding_gradient")
    return out
