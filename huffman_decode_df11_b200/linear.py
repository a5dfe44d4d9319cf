"""The linear product of a model's layer on compressed weights
(df11_decode_linear): y = act(x W^T + bias) * multiplier + residual.

    >>> d = compress_linear(w)                     # once; w is rows x cols, BF16
    >>> y, = decode_linear([d], [x], activations=["silu"], multipliers=[up])
    >>> plan = LinearPlan([q, k, v], [x] * 3, [yq, yk, yv], biases=[bq, bk, bv])
    >>> plan.run()                                 # the same buffers again
"""
from __future__ import annotations

import ctypes
from typing import List, Optional, Sequence

import numpy as np
import torch

from . import (Df11Device, TensorDesc, _check, _one_device, _stream_handle, compress,
               compress_on_device, lib)

# Df11Device.interleave of a weight in the linear product's tile order.  Not a
# row count that interleave_rows takes, so every other product refuses it.
LINEAR_TILES = 16 * 256 + 64
TILE_ROWS, TILE_COLS = 16, 64
LINEAR_MAX_BATCH = 1 << 20

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_TYPES = {torch.bfloat16: 0, torch.float32: 1}


class LinearOp(ctypes.Structure):
    """df11_linear: the linear product applied to one compressed weight."""
    _fields_ = ([(f, ctypes.c_void_p) for f in ("x", "y", "bias", "multiplier", "residual")]
                + [(f, ctypes.c_uint32) for f in ("rows", "cols", "batch", "x_stride", "y_stride",
                                                  "multiplier_stride", "residual_stride")]
                + [(f, ctypes.c_int32) for f in ("activation", "y_type", "bias_type",
                                                 "multiplier_type", "residual_type")])


def _padded(shape):
    rows, cols = shape
    return -(-rows // TILE_ROWS) * TILE_ROWS, -(-cols // TILE_COLS) * TILE_COLS


def tile_linear(w):
    """A rows x cols matrix (array or tensor of 2-byte words) in the linear
    product's tile order, flat: padded with zeros to whole tiles of 16 rows and
    64 columns, and tile after tile along the columns, then down the rows."""
    rows, cols = w.shape
    pr, pc = _padded((rows, cols))
    if isinstance(w, torch.Tensor):
        p = w
        if (pr, pc) != (rows, cols):
            p = torch.zeros(pr, pc, dtype=w.dtype, device=w.device)
            p[:rows, :cols] = w
        v = p.reshape(pr // TILE_ROWS, TILE_ROWS, pc // TILE_COLS, TILE_COLS)
        return v.permute(0, 2, 1, 3).reshape(-1)
    p = np.zeros((pr, pc), w.dtype)
    p[:rows, :cols] = w
    v = p.reshape(pr // TILE_ROWS, TILE_ROWS, pc // TILE_COLS, TILE_COLS).transpose(0, 2, 1, 3)
    return np.ascontiguousarray(v).reshape(-1)


def untile_linear(flat, shape):
    """The inverse of tile_linear: the decoded words of a compressed weight in
    tile order back to its rows x cols matrix."""
    rows, cols = shape
    pr, pc = _padded(shape)
    v = flat.reshape(pr // TILE_ROWS, pc // TILE_COLS, TILE_ROWS, TILE_COLS)
    v = v.permute(0, 2, 1, 3) if isinstance(v, torch.Tensor) else v.transpose(0, 2, 1, 3)
    return v.reshape(pr, pc)[:rows, :cols]


def compress_linear(w, chunk_bytes: int = 24, threads: int = 0, stream=None):
    """Compress a weight (rows x cols BF16) for decode_linear, in its tile
    order.  A CUDA tensor is compressed on its device (compress_on_device) and
    gives a Df11Device; host data are compressed on the host (compress) and
    give a Df11Host, which to_device takes on."""
    if w.ndim != 2 or 0 in w.shape:
        raise ValueError("compress_linear takes a 2-D weight (rows x cols)")
    shape = tuple(int(n) for n in w.shape)
    if isinstance(w, torch.Tensor) and w.is_cuda:
        if stream is None:
            d = compress_on_device(tile_linear(w), chunk_bytes=chunk_bytes)
        else:
            with torch.cuda.stream(stream):
                d = compress_on_device(tile_linear(w), chunk_bytes=chunk_bytes, stream=stream)
    else:
        if isinstance(w, torch.Tensor):
            w = w.detach().contiguous().view(torch.int16).numpy()
        d = compress(tile_linear(np.asarray(w)), chunk_bytes, threads=threads)
    d.shape = shape
    d.interleave = LINEAR_TILES
    return d


def _operand(name, t, shape, device, dtypes):
    """A 1-D or 2-D operand with contiguous rows: (pointer, row stride)."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: expected {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the weight on {device}")
    if t.numel() and shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    stride = t.stride(0) if len(shape) == 2 and shape[0] > 1 else shape[-1]
    if not shape[-1] <= stride < 1 << 32:
        raise ValueError(f"{name}: row stride {stride} below the row's length or too long")
    return t.data_ptr(), stride


def _linear_op(d: Df11Device, x, y, bias, activation, multiplier, residual) -> LinearOp:
    if int(getattr(d, "interleave", 1)) != LINEAR_TILES:
        raise ValueError("decode_linear needs weights compressed by compress_linear")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation {activation!r}: expected one of {', '.join(ACTIVATIONS)}")
    rows, cols = d.shape
    if x.dim() != 2:
        raise ValueError("x must have two dimensions (tokens x cols)")
    tokens, wide = x.shape[0], tuple(_TYPES)
    if tokens > LINEAR_MAX_BATCH:
        raise ValueError(f"at most {LINEAR_MAX_BATCH} tokens per call")
    op = LinearOp(rows=rows, cols=cols, batch=tokens, activation=ACTIVATIONS[activation])
    op.x, op.x_stride = _operand("x", x, (tokens, cols), d.device, (torch.bfloat16, torch.int16))
    op.y, op.y_stride = _operand("y", y, (tokens, rows), d.device, wide)
    op.y_type = _TYPES[y.dtype]
    if bias is not None:
        op.bias, _ = _operand("bias", bias, (rows,), d.device, wide)
        op.bias_type = _TYPES[bias.dtype]
    if multiplier is not None:
        op.multiplier, op.multiplier_stride = _operand("multiplier", multiplier, (tokens, rows),
                                                       d.device, wide)
        op.multiplier_type = _TYPES[multiplier.dtype]
    if residual is not None:
        op.residual, op.residual_stride = _operand("residual", residual, (tokens, rows), d.device,
                                                   wide)
        op.residual_type = _TYPES[residual.dtype]
    return op


def _each(name, values, n, default=None):
    if values is None:
        return [default] * n
    if len(values) != n:
        raise ValueError(f"one {name} (or None) per weight")
    return list(values)


def _aligned_empty(nbytes: int, device) -> torch.Tensor:
    t = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    off = -t.data_ptr() % 256
    return t[off:off + nbytes]


class LinearPlan:
    """The linear products of fixed weights on fixed buffers (a layer's
    projections of one activation buffer, say), prepared once: the arguments
    are checked, the descriptors built and the workspace allocated here, and
    every run() is one library call.

    `xs`: per weight, BF16 activations (tokens x cols); `ys`: float32 or BF16
    outputs (tokens x rows).  `biases` (rows), `multipliers` and `residuals`
    (tokens x rows): per weight a float32 or BF16 tensor or None.
    `activations`: per weight "none", "relu", "gelu", "gelu_tanh" or "silu".
    Rows of all of them must be contiguous; the row strides are free.  A
    residual may be the output itself.  Runs of one plan share its workspace
    and must not overlap on the GPU; plans on several streams at once are
    plans of their own."""

    def __init__(self, ds: Sequence[Df11Device], xs: Sequence[torch.Tensor],
                 ys: Sequence[torch.Tensor], biases=None, activations=None, multipliers=None,
                 residuals=None):
        n = len(ds)
        if not (n == len(xs) == len(ys)):
            raise ValueError("one x and one y per weight")
        bs, acts = _each("bias", biases, n), _each("activation", activations, n, "none")
        ms, rs = _each("multiplier", multipliers, n), _each("residual", residuals, n)
        ops = [_linear_op(*a) for a in zip(ds, xs, ys, bs, acts, ms, rs)]
        self._n = n
        self._keep = (list(ds), list(xs), list(ys), bs, ms, rs)
        self._descs = (TensorDesc * max(n, 1))(*[_weight_desc(d) for d in ds])
        self._ops = (LinearOp * max(n, 1))(*ops)
        self._lib = lib()
        self._device = _one_device(ds) if n else None
        self._work = None
        size = ctypes.c_size_t(0)
        if n:
            with torch.cuda.device(self._device):
                _check(self._lib.df11_linear_workspace(self._descs, self._ops, n,
                                                       ctypes.byref(size)),
                       "df11_linear_workspace")
                self._work = _aligned_empty(size.value, self._device)
        self._bytes = size.value

    @property
    def outs(self) -> List[torch.Tensor]:
        return self._keep[2]

    @property
    def workspace_bytes(self) -> int:
        return self._bytes

    def run(self, err: Optional[torch.Tensor] = None, stream=None) -> List[torch.Tensor]:
        if not self._n:
            return self._keep[2]
        if torch.cuda.current_device() != self._device.index:
            with torch.cuda.device(self._device):
                return self.run(err, stream)
        _check(self._lib.df11_decode_linear(self._descs, self._ops, self._n,
                                            self._work.data_ptr(), self._bytes,
                                            err.data_ptr() if err is not None else None,
                                            _stream_handle(stream)), "df11_decode_linear")
        return self._keep[2]


def _weight_desc(d: Df11Device) -> TensorDesc:
    t = d.desc(torch.empty(0, device=d.device))
    t.out_bf16 = None
    return t


def _on_stream(stream):
    """A torch stream to allocate a call's buffers on (None: the current one)."""
    if stream is None or hasattr(stream, "cuda_stream"):
        return stream
    return torch.cuda.ExternalStream(int(stream))


def decode_linear(ds: Sequence[Df11Device], xs: Sequence[torch.Tensor],
                  ys: Optional[Sequence[torch.Tensor]] = None, biases=None, activations=None,
                  multipliers=None, residuals=None, out_dtype: torch.dtype = torch.bfloat16,
                  err: Optional[torch.Tensor] = None, stream=None) -> List[torch.Tensor]:
    """y = act(x W^T + bias) * multiplier + residual for each weight W
    compressed by compress_linear, decoding W on the way (df11_decode_linear);
    the arguments are LinearPlan's.  Outputs are allocated in `out_dtype` when
    `ys` is None.  Sums run in fp32 and the result is rounded once; the same
    call gives the same bits.  Asynchronous on `stream` (default: the current
    stream); a loop over fixed buffers is cheaper with a LinearPlan."""
    if len(ds) != len(xs):
        raise ValueError("one x per weight")
    if not ds:
        return []
    with torch.cuda.device(ds[0].device), torch.cuda.stream(_on_stream(stream)):
        if ys is None:
            if out_dtype not in _TYPES:
                raise TypeError(f"out_dtype: expected float32 or bfloat16, got {out_dtype}")
            ys = [torch.empty(x.shape[0], d.shape[0], dtype=out_dtype, device=d.device)
                  for d, x in zip(ds, xs)]
        # the workspace is allocated and freed in the order of the call's stream
        return LinearPlan(ds, xs, ys, biases, activations, multipliers, residuals).run(err, stream)
