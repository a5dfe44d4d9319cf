"""Outputs that share memory with what their weight reads are refused, others are not;
without a GPU (beyond 32 tokens the library needs none for the workspace's size)."""
import ctypes
import random

import numpy as np

import huffman_decode_df11_b200 as df11

BASE, OK, INVALID = 1 << 24, 0, 7
ROWS, COLS, TOKENS = 32, 128, 40


def _status(**kw):
    w = df11.LinearWeightDesc(256, 256, 256, 256, df11.LinearParams(ROWS, COLS, 12, 20))
    op = df11.LinearOp(batch=TOKENS, x=BASE, x_stride=COLS, y=BASE + (1 << 22), y_stride=ROWS)
    for k, v in kw.items():
        setattr(op, k, v)
    ws, ops, n = (df11.LinearWeightDesc * 1)(w), (df11.LinearOp * 1)(op), ctypes.c_size_t(0)
    status = df11.lib().df11_linear_workspace(ws, ops, 1, ctypes.byref(n))
    if status == INVALID:  # the call refuses it too, before it looks at a device
        assert df11.lib().df11_decode_linear(ws, ops, 1, BASE, 1 << 40, None, None) == INVALID
        assert n.value == 0
    return status


def test_an_output_on_its_own_operands():
    y = BASE + (1 << 22)
    assert _status() == OK
    assert _status(y=BASE) == INVALID
    assert _status(y=BASE + 2 * COLS * TOKENS - 4, y_type=1) == INVALID     # the last elements of x
    assert _status(y=BASE + 2 * COLS * TOKENS) == OK                        # right behind x
    assert _status(y=BASE, x=BASE + 2 * ROWS * TOKENS) == OK                # right before it
    assert _status(y=BASE, x=BASE + 2 * ROWS * TOKENS - 2) == INVALID
    assert _status(bias=y + 2 * ROWS * TOKENS - 4, bias_type=1) == INVALID
    assert _status(bias=y + 2 * ROWS * TOKENS) == OK
    for name in ("multiplier", "residual"):
        def other(at, stride=ROWS, kind=0):
            return _status(**{name: at, name + "_stride": stride, name + "_type": kind})
        assert other(y) == OK                       # in place
        assert other(y, kind=1) == INVALID          # of another type
        assert other(y, stride=ROWS + 8) == INVALID
        assert other(y + 2) == INVALID              # one element on
        assert other(BASE) == OK                    # on x: both are read
    # no token: nothing is written
    assert _status(batch=0, y=BASE) == OK


def test_columns_of_one_buffer():
    s = COLS + ROWS                                  # elements of BF16 between rows
    assert _status(x_stride=s, y=BASE + 2 * COLS, y_stride=s) == OK
    assert _status(x_stride=s, y=BASE + 2 * COLS - 2, y_stride=s) == INVALID
    assert _status(x=BASE + 2 * ROWS, x_stride=s, y=BASE, y_stride=s) == OK
    assert _status(x=BASE + 2 * ROWS - 2, x_stride=s, y=BASE, y_stride=s) == INVALID
    # the output's rows between those of x, one on: the last one behind the end of x
    assert _status(x_stride=s, y=BASE + 2 * s - 2 * ROWS, y_stride=s) == OK
    assert _status(x_stride=s, y=BASE + 2 * s - 2 * ROWS + 2, y_stride=s) == INVALID


def test_random_places_against_the_bytes():
    rng = random.Random(1)
    seen = {OK: 0, INVALID: 0}
    for _ in range(3000):
        xs, kind = rng.choice([COLS, COLS + ROWS, COLS + 2 * ROWS + 8, 400]), rng.randrange(2)
        size = 4 if kind else 2
        ys = rng.choice([ROWS, xs * 2 // size, xs, 2 * ROWS + 3, 200])
        at = BASE + size * rng.randrange(-ys * TOKENS, xs * TOKENS * 2 // size)
        x = (BASE + 2 * xs * np.arange(TOKENS)[:, None] + np.arange(2 * COLS)).ravel()
        y = (at + size * ys * np.arange(TOKENS)[:, None] + np.arange(size * ROWS)).ravel()
        if ys < ROWS:
            continue
        want = INVALID if np.intersect1d(x, y).size else OK
        seen[want] += 1
        assert _status(x_stride=xs, y=at, y_stride=ys, y_type=kind) == want, (xs, ys, at, kind)
    assert min(seen.values()) > 300
