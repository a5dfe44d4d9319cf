"""Outputs of the embedding's calls on the memory of what they read are refused, without a GPU
(the check stands before the first look at a device)."""
import ctypes

import pytest

import huffman_decode_df11_b200 as df11

AT, ROWS, DIM, TOKENS, INVALID = 1 << 24, 40, 100, 30, 7


def _gradient(**kw):
    op = df11.EmbeddingGradOp(ids=AT, grad=AT + (1 << 20), out=AT + (1 << 21), grad_stride=DIM,
                              out_stride=DIM, rows=ROWS, dim=DIM, tokens=TOKENS, scale=1.0)
    for k, v in kw.items():
        setattr(op, k, v)
    return df11.lib().df11_embedding_gradient(ctypes.byref(op), 256, 1 << 40, None, None)


def _lookup(**kw):
    p = df11.Params(n=ROWS * DIM, total_bits=10000, chunk_bytes=24, threads_per_block=256,
                    num_blocks=1, num_luts=1, max_block_elems=4000, max_len=10,
                    max_chunk_elems=100, max_warp_elems=3000)
    t = df11.TensorDesc(256, 256, 256, 256, 256, 256, 256, None, 256, p)
    op = df11.EmbeddingOp(ids=AT, out=AT + (1 << 20), out_stride=DIM, rows=ROWS, dim=DIM,
                          tokens=TOKENS, scale=1.0)
    for k, v in kw.items():
        setattr(op, k, v)
    return df11.lib().df11_decode_embedding(ctypes.byref(t), ctypes.byref(op), None, None)


@pytest.mark.parametrize("accumulate", [0, 1])
def test_a_gradient_on_what_it_reads(accumulate):
    g, far = AT + (1 << 20), _gradient(accumulate=accumulate)
    assert far not in (0, INVALID)                                   # no device here, or fake memory
    for out in (g, g + 2 * DIM * TOKENS - 2, g - 2 * DIM * ROWS + 2, AT, AT + 4 * TOKENS - 2):
        assert _gradient(out=out, accumulate=accumulate) == INVALID
    for out in (g + 2 * DIM * TOKENS, g - 2 * DIM * ROWS, AT + 4 * TOKENS):
        assert _gradient(out=out, accumulate=accumulate) == far
    assert _gradient(tokens=0, ids=g, grad=g, out=g - 2, accumulate=accumulate) == far  # reads nothing
    # columns of one buffer
    assert _gradient(grad_stride=2 * DIM, out=g + 2 * DIM, out_stride=2 * DIM) == far
    assert _gradient(grad_stride=2 * DIM, out=g + 2 * DIM - 2, out_stride=2 * DIM) == INVALID


def test_a_lookup_on_its_ids():
    far = _lookup()
    assert far not in (0, INVALID)
    assert _lookup(out=AT) == INVALID and _lookup(out=AT + 4 * TOKENS - 2) == INVALID
    assert _lookup(out=AT - 2 * DIM * TOKENS + 2) == INVALID
    assert _lookup(out=AT - 2 * DIM * TOKENS) == far and _lookup(out=AT + 4 * TOKENS) == far
    assert _lookup(ids_type=1, out=AT + 4 * TOKENS) == INVALID
