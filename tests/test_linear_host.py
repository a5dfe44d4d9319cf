"""The linear product's descriptors and refusals, without a GPU."""
import ctypes

import pytest
import torch

import huffman_decode_df11_b200 as df11
from huffman_decode_df11_b200 import linear

FAKE = 1 << 20  # an aligned non-null address; never dereferenced


def test_struct_layout_matches_the_header():
    assert ctypes.sizeof(df11.LinearOp) == 5 * 8 + 5 * 4 + 5 * 4
    assert ctypes.sizeof(df11.LinearParams) == 16
    assert ctypes.sizeof(df11.LinearWeightDesc) == 4 * 8 + 16


def _host_weight(rows=32, cols=128):
    p = df11.LinearParams(rows, cols, 12, 20)
    return df11.LinearWeight(p, torch.zeros(640, dtype=torch.int32),
                             torch.zeros(3, dtype=torch.int32),
                             torch.zeros(rows * cols, dtype=torch.uint8),
                             torch.zeros(linear.LINEAR_TABLE_BYTES, dtype=torch.uint8))


def _bad(match, exc=ValueError, d=None, x=None, y=None, bias=None, act="none", mul=None, res=None):
    d = d or _host_weight()
    x = torch.zeros(4, 128, dtype=torch.bfloat16) if x is None else x
    y = torch.zeros(4, 32) if y is None else y
    with pytest.raises(exc, match=match):
        linear._linear_op(d, x, y, bias, act, mul, res)


def test_refusals_of_the_binding():
    bf = torch.bfloat16
    plain = df11.to_device(df11.compress(torch.randn(32, 128).to(bf)), "cpu", decode_table=False)
    _bad("compress_linear", exc=TypeError, d=plain)
    _bad("activation", act="swish")
    _bad("x", exc=TypeError, x=torch.zeros(4, 128))
    _bad("x must have two", x=torch.zeros(128, dtype=bf))
    _bad("x: expected shape", x=torch.zeros(4, 127, dtype=bf))
    _bad("y", exc=TypeError, y=torch.zeros(4, 32, dtype=torch.float16))
    _bad("y: expected shape", y=torch.zeros(3, 32))
    _bad("rows must be contiguous", y=torch.zeros(32, 4).t())
    _bad("row stride", y=torch.zeros(1, 32).expand(4, 32))
    _bad("bias", bias=torch.zeros(31))
    _bad("bias", exc=TypeError, bias=torch.zeros(32, dtype=torch.float64))
    _bad("multiplier", mul=torch.zeros(4, 31))
    _bad("residual", res=torch.zeros(5, 32))
    with pytest.raises(ValueError):
        df11.compress_linear(torch.zeros(8, dtype=bf))
    with pytest.raises(ValueError):
        df11.compress_linear(torch.zeros(0, 8, dtype=bf))
    with pytest.raises(ValueError):
        df11.LinearPlan([_host_weight()], [], [])
    with pytest.raises(ValueError):
        df11.decode_linear([_host_weight()], [])
    with pytest.raises(TypeError):
        df11.compress_linear(torch.zeros(8, 8))
    tiles = df11.compress(torch.zeros(32, 16, dtype=bf), interleave=16)
    with pytest.raises(ValueError):
        df11.compress_linear(df11.to_device(tiles, "cpu", decode_table=False))


def _weight(**kw):
    w = df11.LinearWeightDesc(FAKE, FAKE, FAKE, FAKE, df11.LinearParams(32, 128, 12, 20))
    for k, v in kw.items():
        setattr(w.params if hasattr(w.params, k) else w, k, v)
    return w


def _op(**kw):
    op = df11.LinearOp(x=FAKE, y=FAKE, batch=4, x_stride=128, y_stride=32)
    for k, v in kw.items():
        setattr(op, k, v)
    return op


def _call(w, op, ws=FAKE, nbytes=1 << 40, err=None):
    return df11.lib().df11_decode_linear((df11.LinearWeightDesc * 1)(w), (df11.LinearOp * 1)(op),
                                         1, ws, nbytes, err, None)


NULL, ALIGN, FORMAT, UNSUPPORTED, TOO_LARGE, INVALID = 1, 2, 3, 4, 6, 7


@pytest.mark.parametrize("status,weight,op", [
    (NULL, {}, dict(x=None)), (NULL, {}, dict(y=None)), (NULL, dict(streams=None), {}),
    (NULL, dict(unit_rows=None), {}), (NULL, dict(table=None), {}),
    (ALIGN, {}, dict(x=FAKE + 1)), (ALIGN, {}, dict(y=FAKE + 1)),
    (ALIGN, {}, dict(y=FAKE + 2, y_type=1)), (ALIGN, {}, dict(bias=FAKE + 2, bias_type=1)),
    (ALIGN, dict(streams=FAKE + 8), {}), (ALIGN, dict(sign_mantissa=FAKE + 8), {}),
    (INVALID, {}, dict(activation=5)), (INVALID, {}, dict(activation=-1)),
    (INVALID, {}, dict(y_type=2)), (INVALID, {}, dict(bias=FAKE, bias_type=7)),
    (INVALID, dict(rows=0), {}), (INVALID, dict(cols=0), {}),
    (INVALID, {}, dict(x_stride=127)), (INVALID, {}, dict(y_stride=31)),
    (INVALID, {}, dict(multiplier=FAKE, multiplier_stride=31)),
    (INVALID, {}, dict(residual=FAKE, residual_stride=0)),
    (TOO_LARGE, {}, dict(batch=(1 << 20) + 1)),
    (TOO_LARGE, dict(rows=1 << 16, cols=1 << 16), dict(x_stride=1 << 16, y_stride=1 << 16)),
    (FORMAT, dict(max_words=0), {}), (FORMAT, dict(max_words=33), {}),
    (FORMAT, dict(stream_rows=25), {}),
])
def test_refusals_of_the_library(status, weight, op):
    assert _call(_weight(**weight), _op(**op)) == status
    n = ctypes.c_size_t(5)
    assert df11.lib().df11_linear_workspace((df11.LinearWeightDesc * 1)(_weight(**weight)),
                                            (df11.LinearOp * 1)(_op(**op)), 1,
                                            ctypes.byref(n)) == status
    assert n.value == 0


def test_empty_calls_do_nothing():
    L = df11.lib()
    assert L.df11_decode_linear(None, None, 0, None, 0, None, None) == 0
    assert L.df11_decode_linear(None, None, 1, None, 0, None, None) == NULL
    assert L.df11_decode_linear(None, None, -1, None, 0, None, None) == INVALID
    assert _call(_weight(), _op(batch=0, x=None, y=None), ws=None, nbytes=0) == 0
    assert L.df11_linear_workspace(None, None, 0, None) == NULL
    assert _call(_weight(), _op(), err=FAKE + 2) == ALIGN


def test_refusals_of_the_builder():
    L, u = df11.lib(), ctypes.c_uint64
    a, b = u(0), u(0)
    assert L.df11_linear_sizes(33, 65, ctypes.byref(a), ctypes.byref(b)) == 0
    assert b.value == 48 * 128 and a.value == 3 + 3
    assert L.df11_linear_sizes(0, 65, ctypes.byref(a), ctypes.byref(b)) == INVALID
    assert L.df11_linear_sizes(1 << 20, 1 << 12, ctypes.byref(a), ctypes.byref(b)) == TOO_LARGE
    assert L.df11_linear_sizes(1, 1, None, ctypes.byref(b)) == NULL
    p = df11.LinearParams()
    ref = ctypes.byref(p)
    assert L.df11_linear_weight_begin(None, 4, 4, FAKE, FAKE, ref, None) == NULL
    assert L.df11_linear_weight_begin(FAKE, 4, 4, FAKE, FAKE, None, None) == NULL
    assert L.df11_linear_weight_begin(FAKE, 4, 0, FAKE, FAKE, ref, None) == INVALID
    assert L.df11_linear_weight_begin(FAKE + 1, 4, 4, FAKE, FAKE, ref, None) == ALIGN
    assert L.df11_linear_weight_begin(FAKE, 4, 4, FAKE, FAKE + 8, ref, None) == ALIGN
    w = _weight()
    assert L.df11_linear_weight_finish(None, ctypes.byref(w), None) == NULL
    assert L.df11_linear_weight_finish(FAKE, None, None) == NULL
    bad = _weight(max_words=99)
    assert L.df11_linear_weight_finish(FAKE, ctypes.byref(bad), None) == FORMAT
    assert L.df11_linear_unpack(ctypes.byref(bad), FAKE, None, None) == FORMAT
    assert L.df11_linear_unpack(ctypes.byref(w), FAKE + 2, None, None) == ALIGN
    assert L.df11_linear_unpack(ctypes.byref(w), None, None, None) == NULL
