"""The linear product's tile order, descriptors and refusals, without a GPU."""
import ctypes

import numpy as np
import pytest
import torch

import huffman_decode_df11_b200 as df11
import oracle
from huffman_decode_df11_b200 import linear

FAKE = 1 << 20  # an aligned non-null address; never dereferenced


@pytest.mark.parametrize("shape", [(1, 1), (16, 64), (17, 65), (37, 131), (48, 640)])
def test_tile_order_is_the_stated_one(shape):
    rows, cols = shape
    w = np.arange(rows * cols, dtype=np.uint16).reshape(shape) + 1
    flat = df11.tile_linear(w)
    pr, pc = -(-rows // 16) * 16, -(-cols // 64) * 64
    assert flat.size == pr * pc
    i = 0
    for rb in range(pr // 16):
        for cg in range(pc // 64):
            for r in range(16 * rb, 16 * rb + 16):
                for c in range(64 * cg, 64 * cg + 64):
                    assert flat[i] == (w[r, c] if r < rows and c < cols else 0)
                    i += 1
    assert np.array_equal(df11.untile_linear(flat, shape), w)
    t = torch.from_numpy(w.view(np.int16))
    assert np.array_equal(df11.tile_linear(t).numpy().view(np.uint16), flat)
    assert torch.equal(df11.untile_linear(df11.tile_linear(t), shape), t)


def test_compressed_on_the_host_decodes_to_the_tiles():
    w = torch.randn(20, 100).to(torch.bfloat16)
    h = df11.compress_linear(w)
    assert h.shape == (20, 100) and h.interleave == df11.LINEAR_TILES and h.n == 32 * 128
    words, _, _ = oracle.decode(h.bitstream, h.code_lengths, h.sign_mantissa, h.n)
    got = df11.untile_linear(words, h.shape)
    assert np.array_equal(got.view(np.int16), w.view(torch.int16).numpy())


def test_struct_layout_matches_the_header():
    assert ctypes.sizeof(df11.LinearOp) == 5 * 8 + 7 * 4 + 5 * 4


def _host_weight(rows=32, cols=128):
    h = df11.compress_linear(torch.randn(rows, cols).to(torch.bfloat16))
    return df11.to_device(h, "cpu", decode_table=False)


def _bad(match, exc=ValueError, d=None, x=None, y=None, bias=None, act="none", mul=None, res=None):
    d = d or _host_weight()
    x = torch.zeros(4, 128, dtype=torch.bfloat16) if x is None else x
    y = torch.zeros(4, 32) if y is None else y
    with pytest.raises(exc, match=match):
        linear._linear_op(d, x, y, bias, act, mul, res)


def test_refusals_of_the_binding():
    bf = torch.bfloat16
    plain = df11.to_device(df11.compress(torch.randn(32, 128).to(bf)), "cpu", decode_table=False)
    _bad("compress_linear", d=plain)
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


def test_tiles_are_refused_by_the_other_products():
    d = _host_weight()
    with pytest.raises(ValueError):
        df11.decode_gemm([d], [torch.zeros(1, 128)], [torch.zeros(1, 32)])
    # an interleave that is no power of two up to 32 is an invalid argument there
    op = df11.GemvOp(FAKE, FAKE, 128, 1, 128, 32, 0, df11.LINEAR_TILES)
    t = d.desc(torch.empty(0))
    assert df11.lib().df11_decode_gemv((df11.TensorDesc * 1)(t), (df11.GemvOp * 1)(op), 1, None,
                                       None) == 7


def _tensor(**kw):
    p = df11.Params(n=32 * 128, total_bits=10000, chunk_bytes=24, threads_per_block=256,
                    num_blocks=1, num_luts=1, max_block_elems=4096, max_len=10,
                    max_chunk_elems=100, max_warp_elems=3000)
    t = df11.TensorDesc(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, p)
    for k, v in kw.items():
        setattr(t.params if hasattr(t.params, k) else t, k, v)
    return t


def _op(**kw):
    op = df11.LinearOp(x=FAKE, y=FAKE, rows=32, cols=128, batch=4, x_stride=128, y_stride=32)
    for k, v in kw.items():
        setattr(op, k, v)
    return op


def _call(t, op, ws=FAKE, nbytes=1 << 40, err=None):
    return df11.lib().df11_decode_linear((df11.TensorDesc * 1)(t), (df11.LinearOp * 1)(op), 1, ws,
                                         nbytes, err, None)


NULL, ALIGN, FORMAT, UNSUPPORTED, TOO_LARGE, INVALID = 1, 2, 3, 4, 6, 7


@pytest.mark.parametrize("status,tensor,op", [
    (NULL, {}, dict(x=None)), (NULL, {}, dict(y=None)), (NULL, dict(bitstream=None), {}),
    (ALIGN, {}, dict(x=FAKE + 1)), (ALIGN, {}, dict(y=FAKE + 1)),
    (ALIGN, {}, dict(y=FAKE + 2, y_type=1)), (ALIGN, {}, dict(bias=FAKE + 2, bias_type=1)),
    (ALIGN, dict(bitstream=FAKE + 8), {}),
    (INVALID, {}, dict(activation=5)), (INVALID, {}, dict(activation=-1)),
    (INVALID, {}, dict(y_type=2)), (INVALID, {}, dict(bias=FAKE, bias_type=7)),
    (INVALID, {}, dict(rows=0)), (INVALID, {}, dict(cols=0)), (INVALID, {}, dict(rows=33)),
    (INVALID, {}, dict(cols=129)), (INVALID, {}, dict(x_stride=127)),
    (INVALID, {}, dict(y_stride=31)),
    (INVALID, {}, dict(multiplier=FAKE, multiplier_stride=31)),
    (INVALID, {}, dict(residual=FAKE, residual_stride=0)),
    (TOO_LARGE, {}, dict(batch=(1 << 20) + 1)), (TOO_LARGE, dict(n=1 << 32), {}),
    (UNSUPPORTED, dict(chunk_counts=None), {}), (UNSUPPORTED, dict(decode_table=None), {}),
    (UNSUPPORTED, dict(chunk_bytes=4, num_blocks=2, max_chunk_elems=30, max_warp_elems=900), {}),
    (FORMAT, dict(num_blocks=2), {}), (FORMAT, dict(max_warp_elems=0), {}),
])
def test_refusals_of_the_library(status, tensor, op):
    assert _call(_tensor(**tensor), _op(**op)) == status
    n = ctypes.c_size_t(5)
    assert df11.lib().df11_linear_workspace((df11.TensorDesc * 1)(_tensor(**tensor)),
                                            (df11.LinearOp * 1)(_op(**op)), 1,
                                            ctypes.byref(n)) == status
    assert n.value == 0


def test_empty_calls_do_nothing():
    L = df11.lib()
    assert L.df11_decode_linear(None, None, 0, None, 0, None, None) == 0
    assert L.df11_decode_linear(None, None, 1, None, 0, None, None) == NULL
    assert L.df11_decode_linear(None, None, -1, None, 0, None, None) == INVALID
    assert _call(_tensor(), _op(batch=0), ws=None, nbytes=0) == 0
    assert L.df11_linear_workspace(None, None, 0, None) == NULL
    assert _call(_tensor(), _op(), err=FAKE + 2) == ALIGN


def test_one_chunk_size_per_call():
    a, b = _tensor(), _tensor(chunk_bytes=8, num_blocks=1, max_chunk_elems=60,
                              max_warp_elems=1900)
    L = df11.lib()
    assert L.df11_decode_linear((df11.TensorDesc * 2)(a, b), (df11.LinearOp * 2)(_op(), _op()), 2,
                                FAKE, 1 << 40, None, None) == INVALID
