"""The linear product on compressed weights (df11_decode_linear) against the
formula in float64 on the original weights.

Tolerances, per output.  z = sum_c w x + b with S = sum_c |w x|.  Products of
BF16 are exact in fp32; the sums run in fp32 on tensor cores, whose additions may
truncate (one unit in the last place, 2^-23 relative, instead of half), in at most
K + 16 additions (K = padded columns; 8 warps' sums, a few thread blocks' and
the bias besides), so
    e1 = (K + 16) 2^-23 (S + |b|).
The activations' slopes are below 1.2 and each is evaluated with a handful of
fp32 operations, 32 half units allowed: e2 = 1.2 e1 + 32 2^-24 |z|.  Multiplier
and residual each add one rounding: e3 = |m| e2 + 2^-23 |a m|,
e4 = e3 + 2^-23 (|a m| + |r|).  The result is rounded once to its type: BF16 by
at most 2^-8 of it, fp32 by 2^-24 (in e4 already).
"""
import math

import numpy as np
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu

df11 = pytest.importorskip("huffman_decode_df11_b200")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.init()


def _bf16(shape, std, seed):
    n = int(np.prod(shape))
    return workloads.gaussian_bf16(n, std, seed).view(torch.bfloat16).view(shape)


def _act64(name, z):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _check(w, x, y, bias=None, activation="none", multiplier=None, residual=None):
    def wide(t):
        return t.detach().cpu().double()
    w, x = wide(w), wide(x)
    K = -(-w.shape[1] // 64) * 64
    z = x @ w.T
    S = x.abs() @ w.abs().T
    if bias is not None:
        z, S = z + wide(bias), S + wide(bias).abs()
    e = (K + 16) * 2.0 ** -23 * S
    a = _act64(activation, z)
    e = 1.2 * e + 32 * 2.0 ** -24 * z.abs()
    if multiplier is not None:
        m = wide(multiplier)
        a = a * m
        e = m.abs() * e + 2.0 ** -23 * a.abs()
    if residual is not None:
        r = wide(residual)
        e = e + 2.0 ** -23 * (a.abs() + r.abs())
        a = a + r
    if y.dtype == torch.bfloat16:
        e = e + 2.0 ** -8 * (a.abs() + e)
    err = (wide(y) - a).abs()
    assert torch.all(err <= e + 1e-38), (float((err - e).max()), float(err.max()))


def _run(ds, xs, **kw):
    err = df11.new_error_word()
    ys = df11.decode_linear(ds, xs, err=err, **kw)
    torch.cuda.synchronize()
    df11.check_device_error(err)
    return ys


SIZES = [(16, 64, 1), (1, 1, 1), (37, 131, 3), (1000, 2048, 8), (4096, 4096, 1), (777, 1411, 9),
         (512, 12288, 17), (300, 400, 32), (33, 48, 33), (1013, 1411, 77), (256, 256, 128),
         (130, 640, 129), (1024, 4096, 300), (520, 64, 1000), (2048, 1024, 24), (4100, 96, 5)]


@pytest.mark.parametrize("rows,cols,tokens", SIZES)
def test_product_alone(rows, cols, tokens):
    w = _bf16((rows, cols), cols ** -0.5, rows + cols)
    x = _bf16((tokens, cols), 1.0, tokens + cols).cuda()
    d = df11.compress_linear(w.cuda())
    for dtype in (torch.float32, torch.bfloat16):
        y, = _run([d], [x], out_dtype=dtype)
        assert y.dtype == dtype
        _check(w, x, y)


@pytest.mark.parametrize("chunk_bytes", [8, 16, 24])
@pytest.mark.parametrize("tokens", [1, 12, 30, 40])
def test_chunk_sizes(chunk_bytes, tokens):
    w = _bf16((200, 1000), 0.02, 3)
    x = _bf16((tokens, 1000), 1.0, 4).cuda()
    y, = _run([df11.compress_linear(w.cuda(), chunk_bytes)], [x], out_dtype=torch.float32)
    _check(w, x, y)


@pytest.mark.parametrize("activation", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("tokens", [2, 70])
@pytest.mark.parametrize("rows", [320, 333])
@pytest.mark.parametrize("extras", [torch.float32, torch.bfloat16])
def test_epilogue(activation, tokens, rows, extras):
    cols = 192
    g = torch.Generator().manual_seed(rows + tokens)
    w = _bf16((rows, cols), 0.2, 8)
    x = _bf16((tokens, cols), 1.0, 9).cuda()
    b = torch.randn(rows, generator=g).to(extras).cuda()
    m = torch.randn(tokens, rows, generator=g).to(extras).cuda()
    r = torch.randn(tokens, rows, generator=g).to(extras).cuda()
    d = df11.compress_linear(w.cuda())
    for bias, mul, res in ((b, m, r), (b, None, None), (None, m, None), (None, None, r)):
        for dtype in (torch.float32, torch.bfloat16):
            y, = _run([d], [x], biases=[bias], activations=[activation], multipliers=[mul],
                      residuals=[res], out_dtype=dtype)
            _check(w, x, y, bias, activation, mul, res)


@pytest.mark.parametrize("tokens", [1, 8, 9, 16, 17, 32, 33, 128, 129])
def test_token_counts_around_the_variants(tokens):
    w = _bf16((160, 448), 0.05, 1)
    x = _bf16((tokens, 448), 1.0, 2).cuda()
    y, = _run([df11.compress_linear(w.cuda())], [x], out_dtype=torch.float32)
    _check(w, x, y)


@pytest.mark.parametrize("tokens", [3, 50])
def test_strides_and_bytes_around_the_rows(tokens):
    rows, cols = 130, 200
    w = _bf16((rows, cols), 0.1, 1)
    xs = _bf16((tokens + 1, cols + 7), 1.0, 2).cuda()
    x = xs[1:, 3:cols + 3]                          # odd stride, misaligned base
    yb = torch.full((tokens + 2, rows + 9), 7.0, device="cuda")
    y = yb[1:tokens + 1, 4:rows + 4]
    rb = torch.randn(tokens, rows + 3, device="cuda")
    r = rb[:, :rows]
    d = df11.compress_linear(w.cuda())
    _run([d], [x], ys=[y], residuals=[r])
    _check(w, x, y, residual=r)
    yb[1:tokens + 1, 4:rows + 4] = 7.0
    assert torch.all(yb == 7.0)                     # nothing else was written


@pytest.mark.parametrize("tokens", [4, 64])
def test_residual_in_place(tokens):
    w = _bf16((128, 256), 0.1, 1)
    x = _bf16((tokens, 256), 1.0, 2).cuda()
    r = _bf16((tokens, 128), 1.0, 3).cuda()
    y = r.clone()
    _run([df11.compress_linear(w.cuda())], [x], ys=[y], residuals=[y])
    _check(w, x, y, residual=r)


@pytest.mark.parametrize("tokens", [1, 6, 31, 90])
def test_several_weights_in_one_call(tokens):
    shapes = [(256, 512), (64, 512), (65, 512), (31, 100), (1, 512)] * 4   # 20: two launches
    ws = [_bf16(s, 0.1, 30 + i) for i, s in enumerate(shapes)]
    xs = [_bf16((tokens, s[1]), 1.0, 60 + i).cuda() for i, s in enumerate(shapes)]
    ys = _run([df11.compress_linear(w.cuda()) for w in ws], xs, out_dtype=torch.float32)
    for w, x, y in zip(ws, xs, ys):
        _check(w, x, y)


def test_tokens_differ_within_a_call_and_none():
    ws = [_bf16((96, 128), 0.1, i) for i in range(4)]
    xs = [_bf16((t, 128), 1.0, 9 + t).cuda() for t in (1, 0, 30, 5)]
    ds = [df11.compress_linear(w.cuda()) for w in ws]
    for group in (slice(0, 4), slice(1, 2)):
        ys = _run(ds[group], xs[group], out_dtype=torch.float32)
        for w, x, y in zip(ws[group], xs[group], ys):
            assert y.shape == (x.shape[0], 96)
            _check(w, x, y)
    assert df11.decode_linear([], []) == []


def _words(kind, n):
    if kind == "one exponent":          # a one-bit code: the most elements per chunk
        g = torch.Generator().manual_seed(1)
        return torch.where(torch.rand(n, generator=g) < 0.5, 1.0, -1.5).to(torch.bfloat16)
    return workloads.adversarial_mix(n, seed=5).view(torch.bfloat16)


@pytest.mark.parametrize("kind", ["one exponent", "mix"])
@pytest.mark.parametrize("tokens", [1, 20, 40])
def test_other_exponent_distributions(kind, tokens):
    rows, cols = 208, 1280
    w = _words(kind, rows * cols).view(rows, cols)
    x = _bf16((tokens, cols), 1.0, 2).cuda()
    y, = _run([df11.compress_linear(w.cuda())], [x], out_dtype=torch.float32)
    _check(w, x, y)


@pytest.mark.parametrize("tokens", [1, 24, 100])
def test_zero_weights_and_signs(tokens):
    w = torch.zeros(48, 64, dtype=torch.bfloat16)
    w[5, 7] = -2.0
    x = _bf16((tokens, 64), 1.0, 2).cuda()
    y, = _run([df11.compress_linear(w.cuda())], [x], out_dtype=torch.float32)
    _check(w, x, y)
    assert torch.count_nonzero(y[:, [r for r in range(48) if r != 5]]) == 0


@pytest.mark.parametrize("tokens", [2, 40])
def test_nan_of_one_token_or_weight_stays_there(tokens):
    w = _bf16((64, 128), 0.1, 1)
    w[9, 100] = float("nan")
    x = _bf16((tokens, 128), 1.0, 2)
    x[1, 3] = float("nan")
    y, = _run([df11.compress_linear(w.cuda())], [x.cuda()], out_dtype=torch.float32)
    y = y.cpu()
    assert torch.isnan(y[1]).all() and torch.isnan(y[:, 9]).all()
    keep = [r for r in range(64) if r != 9]
    tk = [t for t in range(tokens) if t != 1]
    assert torch.isfinite(y[tk][:, keep]).all()


@pytest.mark.parametrize("tokens", [1, 7, 16, 32, 200])
def test_a_call_repeats_bit_for_bit(tokens):
    w = _bf16((1024, 2048), 0.02, 1)
    x = _bf16((tokens, 2048), 1.0, 2).cuda()
    d = df11.compress_linear(w.cuda())
    first = _run([d], [x], out_dtype=torch.float32)[0].clone()
    for _ in range(5):
        assert torch.equal(_run([d], [x], out_dtype=torch.float32)[0], first)


@pytest.mark.parametrize("tokens", [3, 48])
def test_captured_graphs_and_a_side_stream(tokens):
    w = _bf16((512, 768), 0.05, 1)
    d = df11.compress_linear(w.cuda())
    x = _bf16((tokens, 768), 1.0, 2).cuda()
    y = torch.empty(tokens, 512, device="cuda")
    plan = df11.LinearPlan([d], [x], [y], activations=["silu"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        plan.run()
        graphs = []
        for _ in range(2):           # two graphs of one plan, replayed one after the other
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                plan.run()
            graphs.append(g)
        for i, g in enumerate(graphs * 2):
            x.copy_(_bf16((tokens, 768), 1.0, 50 + i))
            g.replay()
            side.synchronize()
            _check(w, x, y, activation="silu")
    # an explicit stream that is not the current one, by handle
    x2 = _bf16((tokens, 768), 1.0, 99).cuda()
    torch.cuda.synchronize()
    y2, = df11.decode_linear([d], [x2], stream=side.cuda_stream, out_dtype=torch.float32)
    side.synchronize()
    _check(w, x2, y2)


def test_two_plans_at_once_on_two_streams():
    w = _bf16((1024, 1024), 0.03, 1)
    d = df11.compress_linear(w.cuda())
    xs = [_bf16((t, 1024), 1.0, 7 + t).cuda() for t in (2, 64)]
    plans = [df11.LinearPlan([d], [x], [torch.empty(x.shape[0], 1024, device="cuda")]) for x in xs]
    streams = [torch.cuda.Stream() for _ in plans]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, s in zip(plans, streams):
            p.run(stream=s)
    torch.cuda.synchronize()
    for p, x in zip(plans, xs):
        _check(w, x, p.outs[0])


@pytest.mark.parametrize("tokens", [4, 40])
def test_corrupt_counts_are_flagged_and_the_next_call_is_right(tokens):
    w = _bf16((256, 1024), 0.03, 1)
    d = df11.compress_linear(w.cuda())
    x = _bf16((tokens, 1024), 1.0, 2).cuda()
    good = int(d.chunk_counts[40])
    d.chunk_counts[40] = good + 1
    err = df11.new_error_word()
    df11.decode_linear([d], [x], err=err)
    torch.cuda.synchronize()
    with pytest.raises(df11.Df11Error):
        df11.check_device_error(err)
    d.chunk_counts[40] = good
    y, = _run([d], [x], out_dtype=torch.float32)
    _check(w, x, y)


def test_decoding_the_tiles_gives_the_weight_back():
    w = _bf16((77, 150), 0.03, 1)
    d = df11.compress_linear(w.cuda())
    out = df11.decode(d)
    assert torch.equal(df11.untile_linear(out.view(torch.int16), (77, 150)).cpu(),
                       w.view(torch.int16))
    h = df11.compress_linear(w)                       # on the host: the same tensor
    assert h.shape == (77, 150) and h.interleave == df11.LINEAR_TILES
    assert np.array_equal(h.bitstream, d.bitstream.cpu().numpy())
    y, = _run([df11.to_device(h)], [_bf16((2, 150), 1.0, 5).cuda()])
    _check(w, _bf16((2, 150), 1.0, 5), y)
