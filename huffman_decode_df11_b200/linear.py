"""The linear product of a model's layer on compressed weights
(df11_decode_linear): y = act(x W^T + bias) * multiplier + residual.

    >>> d = compress_linear(w)                     # once; w is rows x cols, BF16
    >>> y, = decode_linear([d], [x], activations=["silu"], multipliers=[up])
    >>> plan = LinearPlan([q, k, v], [x] * 3, [yq, yk, yv], biases=[bq, bk, bv])
    >>> plan.run()                                 # the same buffers again
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import List, Optional, Sequence, Union

import numpy as np
import torch

from . import Df11Device, Df11Host, _check, _one_device, _stream_handle, decode, lib, to_device

TILE_ROWS, TILE_COLS, UNIT_TILES = 16, 64, 4
LINEAR_TABLE_BYTES = 4 * 256 + 256 + 256
LINEAR_MAX_BATCH = 1 << 20

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_TYPES = {torch.bfloat16: 0, torch.float32: 1}
_INVALID = 7  # DF11_ERR_INVALID


class LinearParams(ctypes.Structure):
    """df11_linear_params: shape and layout of a weight for the linear product."""
    _fields_ = [(f, ctypes.c_uint32) for f in ("rows", "cols", "max_words", "stream_rows")]


class LinearWeightDesc(ctypes.Structure):
    """df11_linear_weight: device pointers of a weight and its parameters."""
    _fields_ = [("streams", ctypes.c_void_p), ("unit_rows", ctypes.c_void_p),
                ("sign_mantissa", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("params", LinearParams)]


class LinearOp(ctypes.Structure):
    """df11_linear: the linear product applied to one compressed weight."""
    _fields_ = ([(f, ctypes.c_void_p) for f in ("x", "y", "bias", "multiplier", "residual")]
                + [(f, ctypes.c_uint32) for f in ("batch", "x_stride", "y_stride",
                                                  "multiplier_stride", "residual_stride")]
                + [(f, ctypes.c_int32) for f in ("activation", "y_type", "bias_type",
                                                 "multiplier_type", "residual_type")])


@dataclass
class LinearWeight:
    """A weight (rows x cols) compressed for the linear product, in device
    memory (compress_linear)."""
    params: LinearParams
    streams: torch.Tensor        # int32: the units' 32 bitstreams, word by word
    unit_rows: torch.Tensor      # int32: first row of 32 words of each unit, and the total
    sign_mantissa: torch.Tensor  # uint8, padded rows x padded columns
    table: torch.Tensor          # uint8: decode table

    @property
    def shape(self) -> tuple:
        return int(self.params.rows), int(self.params.cols)

    @property
    def device(self):
        return self.streams.device

    def compressed_bytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in
                   (self.streams, self.unit_rows, self.sign_mantissa, self.table))

    def to(self, device) -> "LinearWeight":
        """The same weight with its buffers on `device` (host memory to keep it, say)."""
        return LinearWeight(LinearParams.from_buffer_copy(self.params),
                            *[t.to(device) for t in (self.streams, self.unit_rows,
                                                     self.sign_mantissa, self.table)])

    def desc(self) -> LinearWeightDesc:
        return LinearWeightDesc(self.streams.data_ptr(), self.unit_rows.data_ptr(),
                                self.sign_mantissa.data_ptr(), self.table.data_ptr(), self.params)


def compress_linear(w: Union[torch.Tensor, Df11Device, Df11Host], device=None,
                    stream=None) -> LinearWeight:
    """Compress a weight (rows x cols) for decode_linear, on the device
    (df11_linear_weight_begin / _finish).  `w`: BF16 words (bfloat16, int16 or
    uint16) in device or host memory, or a row-major compressed tensor (decoded on
    the way); data in host memory go to `device` (default: the current CUDA device)
    first.  Lossless, like every form of the format; decode_weight gives
    the words back.  Synchronises the stream."""
    with torch.cuda.stream(_on_stream(stream)):
        if isinstance(w, Df11Host):
            w = to_device(w, device or "cuda")
        if isinstance(w, Df11Device):
            if len(w.shape) != 2 or int(getattr(w, "interleave", 1)) != 1:
                raise ValueError("compress_linear takes a 2-D weight (rows x cols), row-major")
            with torch.cuda.device(w.device):
                w = decode(w).view(w.shape)
        if not isinstance(w, torch.Tensor):
            w = torch.from_numpy(np.ascontiguousarray(w).view(np.int16))
        if w.dim() != 2 or 0 in w.shape:
            raise ValueError("compress_linear takes a 2-D weight (rows x cols)")
        if w.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
            raise TypeError(f"expected BF16 words (bfloat16, int16 or uint16), got {w.dtype}")
        if not w.is_cuda:
            w = w.detach().to(device or "cuda")
        with torch.cuda.device(w.device):
            return _compress_linear(w.detach().contiguous(), stream)


def _compress_linear(w: torch.Tensor, stream) -> LinearWeight:
    rows, cols = w.shape
    L, sh, dev = lib(), _stream_handle(stream), w.device
    if rows >= 1 << 32 or cols >= 1 << 32:
        raise ValueError("weight too large")
    units, sm = ctypes.c_uint64(0), ctypes.c_uint64(0)
    _check(L.df11_linear_sizes(rows, cols, ctypes.byref(units), ctypes.byref(sm)),
           "df11_linear_sizes")
    p = LinearParams()
    unit_rows = torch.empty(units.value, dtype=torch.int32, device=dev)
    table = torch.empty(LINEAR_TABLE_BYTES, dtype=torch.uint8, device=dev)
    _check(L.df11_linear_weight_begin(w.data_ptr(), rows, cols, unit_rows.data_ptr(),
                                      table.data_ptr(), ctypes.byref(p), sh),
           "df11_linear_weight_begin")
    per_row = -(-cols // (TILE_COLS * UNIT_TILES))
    out = LinearWeight(
        params=p, streams=torch.empty(p.stream_rows * 32, dtype=torch.int32, device=dev),
        unit_rows=unit_rows[: -(-rows // TILE_ROWS) * per_row + 1].clone(),
        sign_mantissa=torch.empty(sm.value, dtype=torch.uint8, device=dev), table=table)
    d = out.desc()
    _check(L.df11_linear_weight_finish(w.data_ptr(), ctypes.byref(d), sh),
           "df11_linear_weight_finish")
    torch.cuda.current_stream().synchronize()
    return out


def decode_weight(d: LinearWeight, err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The BF16 matrix (rows x cols) of a weight compressed by compress_linear, bit for
    bit (df11_linear_unpack).  Asynchronous on `stream` (default: the current stream)."""
    rows, cols = d.shape
    pr, pc = -(-rows // TILE_ROWS) * TILE_ROWS, -(-cols // TILE_COLS) * TILE_COLS
    with torch.cuda.device(d.device), torch.cuda.stream(_on_stream(stream)):
        tiles = torch.empty(pr * pc, dtype=torch.bfloat16, device=d.device)
        desc = d.desc()
        _check(lib().df11_linear_unpack(ctypes.byref(desc), tiles.data_ptr(),
                                        err.data_ptr() if err is not None else None,
                                        _stream_handle(stream)), "df11_linear_unpack")
        v = tiles.view(pr // TILE_ROWS, pc // TILE_COLS, TILE_ROWS, TILE_COLS)
        return v.permute(0, 2, 1, 3).reshape(pr, pc)[:rows, :cols].contiguous()


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


def _linear_op(d: LinearWeight, x, y, bias, activation, multiplier, residual) -> LinearOp:
    if not isinstance(d, LinearWeight):
        raise TypeError("decode_linear needs weights compressed by compress_linear")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation {activation!r}: expected one of {', '.join(ACTIVATIONS)}")
    rows, cols = d.shape
    if x.dim() != 2:
        raise ValueError("x must have two dimensions (tokens x cols)")
    tokens, wide = x.shape[0], tuple(_TYPES)
    if tokens > LINEAR_MAX_BATCH:
        raise ValueError(f"at most {LINEAR_MAX_BATCH} tokens per call")
    op = LinearOp(batch=tokens, activation=ACTIVATIONS[activation])
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
    return t[off:] if off else t  # allocations start on 256 bytes as a rule


class LinearPlan:
    """The linear products of fixed weights on fixed buffers (a layer's
    projections of one activation buffer, say), prepared once: the arguments
    are checked, the descriptors built and the workspace allocated here, and
    every run() is one library call.

    `xs`: per weight, BF16 activations (tokens x cols); `ys`: float32 or BF16
    outputs (tokens x rows).  `biases` (rows), `multipliers` and `residuals`
    (tokens x rows): per weight a float32 or BF16 tensor or None.
    `activations`: per weight "none", "relu", "gelu", "gelu_tanh" or "silu".
    Rows of all of them must be contiguous, at any distance of a row's length
    or more.  A multiplier or a residual may be the output itself (the same rows and
    type); otherwise no output may share memory with what its own weight reads (refused) or
    another one does, since they run at the same time.  Runs of one plan share its
    workspace and must not overlap on the GPU, graphs that captured them
    included; for several streams at once, make a plan for each.  The first run on a
    stream other than the one the plan was made on, or a captured one, is ordered
    behind the work that was queued there by then (the workspace's memory may have
    been in use by it).  A graph that captured a run keeps neither the plan nor its
    workspace alive: the plan has to outlive the graph, like the buffers.  Beyond 32
    tokens the workspace holds the decoded weights, two bytes each (workspace_bytes);
    decode_linear allocates it for the call only."""

    def __init__(self, ds: Sequence[LinearWeight], xs: Sequence[torch.Tensor],
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
        self._descs = (LinearWeightDesc * max(n, 1))(*[d.desc() for d in ds])
        self._ops = (LinearOp * max(n, 1))(*ops)
        self._lib = lib()
        self._device = _one_device(ds) if n else None
        self._work = None
        size = ctypes.c_size_t(0)
        if n:
            with torch.cuda.device(self._device):
                status = self._lib.df11_linear_workspace(self._descs, self._ops, n,
                                                         ctypes.byref(size))
                if status == _INVALID:  # what is left of that after _linear_op
                    raise ValueError("an output shares memory with its weight's x, bias, "
                                     "multiplier or residual")
                _check(status, "df11_linear_workspace")
                self._work = _aligned_empty(size.value, self._device)
                self._streams = {_stream_handle(None)}  # ordered behind, and known to the allocator
                self._mark()
        self._bytes = size.value

    _born = None

    def _mark(self):
        """An event behind all that may still use the workspace's memory as somebody else's,
        until that is known to be done.  Not external in a capture: only its own streams
        can wait for it, and later runs are the graph's users' to order."""
        self._capture = self._lib.df11_capture_id(_stream_handle(None))
        self._born = torch.cuda.Event(external=not self._capture)
        self._born.record()
        self._event = self._born  # a graph's wait names it for as long as the graph lives

    @property
    def outs(self) -> List[torch.Tensor]:
        return self._keep[2]

    @property
    def workspace_bytes(self) -> int:
        return self._bytes

    def _enter(self, handle):
        """What a run on a stream needs before it, as long as anything does."""
        s, capture = _on_stream(handle), self._lib.df11_capture_id(handle)
        if self._born is not None and (capture != self._capture if self._capture else
                                       self._lib.df11_event_done(self._born.cuda_event) == 1):
            self._born = None  # over, for every stream and graph
        # a graph may be replayed on any stream, so a captured run waits by itself
        if self._born is not None and (handle not in self._streams or
                                       capture and not self._capture):
            s.wait_event(self._born)
        if not capture and handle not in self._streams:
            # a plan dropped while it runs there keeps its workspace until that is done
            self._work.record_stream(s)
            self._streams.add(handle)

    def run(self, err: Optional[torch.Tensor] = None, stream=None) -> List[torch.Tensor]:
        if not self._n:
            return self._keep[2]
        if torch.cuda.current_device() != self._device.index:
            with torch.cuda.device(self._device):
                return self.run(err, stream)
        handle = _stream_handle(stream)
        if self._born is not None or handle not in self._streams:
            self._enter(handle)
        _check(self._lib.df11_decode_linear(self._descs, self._ops, self._n,
                                            self._work.data_ptr(), self._bytes,
                                            err.data_ptr() if err is not None else None, handle),
               "df11_decode_linear")
        return self._keep[2]


class _OneRun(LinearPlan):
    """A plan that runs once, on the stream it is made on."""

    def _mark(self):
        pass


def _on_stream(stream):
    """A torch stream to allocate a call's buffers on (None: the current one)."""
    if stream is None or hasattr(stream, "cuda_stream"):
        return stream
    return torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()


def decode_linear(ds: Sequence[LinearWeight], xs: Sequence[torch.Tensor],
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
        return _OneRun(ds, xs, ys, biases, activations, multipliers, residuals).run(err, stream)
