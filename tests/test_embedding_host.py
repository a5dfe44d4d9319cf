"""The embedding's descriptors and refusals, without a GPU."""
import ctypes

import pytest
import torch

import huffman_decode_df11_b200 as df11
from huffman_decode_df11_b200 import embedding

FAKE = 1 << 20  # an aligned non-null address; never dereferenced
NULL, ALIGN, FORMAT, UNSUPPORTED, TOO_LARGE, INVALID = 1, 2, 3, 4, 6, 7


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(df11.EmbeddingOp) == 2 * 8 + 8 + 3 * 4 + 2 * 4 + 4
    assert ctypes.sizeof(df11.EmbeddingGradOp) == 3 * 8 + 2 * 8 + 3 * 4 + 4 * 4 + 4


def _tensor(**kw):
    p = df11.Params(n=40 * 100, total_bits=10000, chunk_bytes=24, threads_per_block=256,
                    num_blocks=1, num_luts=1, max_block_elems=4000, max_len=10,
                    max_chunk_elems=100, max_warp_elems=3000)
    t = df11.TensorDesc(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, p)
    for k, v in kw.items():
        setattr(t.params if hasattr(t.params, k) else t, k, v)
    return t


def _lookup(**kw):
    op = df11.EmbeddingOp(ids=FAKE, out=FAKE, out_stride=100, rows=40, dim=100, tokens=3,
                          scale=1.0)
    for k, v in kw.items():
        setattr(op, k, v)
    return op


@pytest.mark.parametrize("status,tensor,op", [
    (NULL, {}, dict(ids=None)), (NULL, {}, dict(out=None)), (NULL, dict(gaps=None), {}),
    (ALIGN, {}, dict(ids=FAKE + 2)), (ALIGN, {}, dict(ids=FAKE + 4, ids_type=1)),
    (ALIGN, {}, dict(out=FAKE + 1)), (ALIGN, {}, dict(out=FAKE + 2, out_type=1)),
    (ALIGN, dict(sign_mantissa=FAKE + 4), {}),
    (INVALID, {}, dict(rows=39)), (INVALID, {}, dict(rows=0)), (INVALID, {}, dict(dim=0)),
    (INVALID, {}, dict(out_stride=99)), (INVALID, {}, dict(ids_type=2)),
    (INVALID, {}, dict(out_type=-1)),
    (TOO_LARGE, {}, dict(tokens=1 << 31)), (TOO_LARGE, dict(n=1 << 32), {}),
    (UNSUPPORTED, dict(chunk_counts=None), {}), (UNSUPPORTED, dict(decode_table=None), {}),
    (FORMAT, dict(num_blocks=2), {}),
])
def test_lookup_refusals_of_the_library(status, tensor, op):
    t, o = _tensor(**tensor), _lookup(**op)
    assert df11.lib().df11_decode_embedding(ctypes.byref(t), ctypes.byref(o), None, None) == status


def test_lookup_of_nothing():
    L, t, o = df11.lib(), _tensor(), _lookup()
    assert L.df11_decode_embedding(None, ctypes.byref(o), None, None) == NULL
    assert L.df11_decode_embedding(ctypes.byref(t), None, None, None) == NULL
    assert L.df11_decode_embedding(ctypes.byref(t), ctypes.byref(o), FAKE + 2, None) == ALIGN
    none = _lookup(tokens=0, ids=None, out=None)
    assert L.df11_decode_embedding(ctypes.byref(t), ctypes.byref(none), None, None) == 0


def _gradient(**kw):
    op = df11.EmbeddingGradOp(ids=FAKE, grad=FAKE, out=FAKE, grad_stride=100, out_stride=100,
                              rows=40, dim=100, tokens=3, scale=1.0)
    for k, v in kw.items():
        setattr(op, k, v)
    return op


@pytest.mark.parametrize("status,op", [
    (NULL, dict(ids=None)), (NULL, dict(grad=None)), (NULL, dict(out=None)),
    (ALIGN, dict(ids=FAKE + 2)), (ALIGN, dict(ids=FAKE + 4, ids_type=1)),
    (ALIGN, dict(grad=FAKE + 1)), (ALIGN, dict(grad=FAKE + 2, grad_type=1)),
    (ALIGN, dict(out=FAKE + 2, out_type=1)),
    (INVALID, dict(rows=0)), (INVALID, dict(dim=0)), (INVALID, dict(grad_stride=99)),
    (INVALID, dict(out_stride=99)), (INVALID, dict(ids_type=5)), (INVALID, dict(grad_type=3)),
    (INVALID, dict(out_type=3)),
    (TOO_LARGE, dict(rows=1 << 31)), (TOO_LARGE, dict(tokens=1 << 31)),
])
def test_gradient_refusals_of_the_library(status, op):
    L, o, n = df11.lib(), _gradient(**op), ctypes.c_size_t(3)
    assert L.df11_embedding_gradient(ctypes.byref(o), FAKE, 1 << 40, None, None) == status
    assert L.df11_embedding_gradient_workspace(ctypes.byref(o), ctypes.byref(n)) == status
    assert n.value == 0


def test_gradient_workspace():
    L, o, n = df11.lib(), _gradient(), ctypes.c_size_t(0)
    assert L.df11_embedding_gradient_workspace(ctypes.byref(o), ctypes.byref(n)) == 0
    assert n.value > 0
    assert L.df11_embedding_gradient_workspace(ctypes.byref(o), None) == NULL
    assert L.df11_embedding_gradient(None, FAKE, 1, None, None) == NULL
    assert L.df11_embedding_gradient(ctypes.byref(o), None, 1 << 30, None, None) == NULL
    assert L.df11_embedding_gradient(ctypes.byref(o), FAKE + 128, 1 << 30, None, None) == ALIGN
    assert L.df11_embedding_gradient(ctypes.byref(o), FAKE, n.value - 1, None, None) == INVALID
    assert L.df11_embedding_gradient(ctypes.byref(o), FAKE, n.value, FAKE + 1, None) == ALIGN


def test_refusals_of_the_binding():
    bf = torch.bfloat16
    w = torch.randn(40, 100).to(bf)
    d = df11.to_device(df11.compress(w), "cpu", decode_table=False)
    ids, out = torch.zeros(3, dtype=torch.int64), torch.zeros(3, 100)

    def bad(exc, match, d=d, ids=ids, out=out, scale=1.0):
        with pytest.raises(exc, match=match):
            embedding._embedding_op(d, ids, out, scale)

    rows = df11.compress(torch.randn(32, 64).to(bf), interleave=16)
    bad(ValueError, "row-major", d=df11.to_device(rows, "cpu", decode_table=False))
    flat = df11.to_device(df11.compress(w.view(-1)), "cpu", decode_table=False)
    bad(ValueError, "2-D", d=flat)
    bad(TypeError, "ids", ids=ids.to(torch.int16))
    bad(ValueError, "contiguous", ids=torch.zeros(6, dtype=torch.int64)[::2])
    bad(TypeError, "out", out=out.half())
    bad(ValueError, "out", out=torch.zeros(3, 99))
    bad(ValueError, "out", out=torch.zeros(2, 100))
    bad(ValueError, "rows", out=torch.zeros(100, 3).t())
    bad(ValueError, "scale", scale=float("inf"))
    with pytest.raises(ValueError, match="CUDA"):
        df11.embedding_gradient(ids, out, 40)
    with pytest.raises(TypeError, match="grad"):
        df11.embedding_gradient(ids, out.half(), 40)
