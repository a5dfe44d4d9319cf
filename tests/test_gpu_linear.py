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
         (130, 640, 129), (1024, 4096, 300), (520, 64, 1000), (2048, 1024, 24), (4100, 96, 5),
         (20000, 64, 2), (40, 20000, 3), (5000, 300, 33), (16, 40000, 20), (530, 260, 32)]


@pytest.mark.parametrize("rows,cols,tokens", SIZES)
def test_product_alone(rows, cols, tokens):
    w = _bf16((rows, cols), cols ** -0.5, rows + cols)
    x = _bf16((tokens, cols), 1.0, tokens + cols).cuda()
    d = df11.compress_linear(w.cuda())
    for dtype in (torch.float32, torch.bfloat16):
        y, = _run([d], [x], out_dtype=dtype)
        assert y.dtype == dtype
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


@pytest.mark.parametrize("tokens", [2, 40])
def test_infinities_follow_the_formula(tokens):
    # an infinite activation reaches every output of its token with the sign of its weight,
    # NaN where the weight is zero, and no other token
    w = _bf16((80, 200), 0.1, 1)
    w[7, 130] = 0.0
    x = _bf16((tokens, 200), 1.0, 2)
    x[1, 130] = float("inf")
    y, = _run([df11.compress_linear(w.cuda())], [x.cuda()], out_dtype=torch.float32)
    y = y.cpu()
    assert torch.isnan(y[1, 7])
    rest = [r for r in range(80) if r != 7]
    assert torch.equal(y[1, rest], torch.sign(w[rest, 130].float()) * float("inf"))
    assert torch.isfinite(y[[t for t in range(tokens) if t != 1]]).all()


def _lane_streams(w):
    """The streams of a compressed weight decoded one codeword at a time, in plain
    Python: the words (padded rows x padded columns) they stand for."""
    p = w.params
    rows, cols = -(-p.rows // 16) * 16, -(-p.cols // 64) * 64
    words = w.streams.cpu().numpy().view(np.uint32).reshape(-1, 32)
    first = w.unit_rows.cpu().numpy()
    sm = w.sign_mantissa.cpu().numpy().view(np.uint32).reshape(rows // 16, cols // 64, 2, 32, 4)
    mantissa, sign = (0, 16, 8, 24), (15, 31, 23, 7)
    # the code, from its stored codewords and lengths
    tail = w.table.cpu().numpy()[-512:]
    book = {f"{int(tail[e]):b}".zfill(int(tail[256 + e]))[::-1]: e
            for e in range(256) if tail[256 + e]}
    out = np.zeros((rows, cols), np.uint16)
    per_row = -(-cols // 256)
    assert len(first) == rows // 16 * per_row + 1 and first[-1] == p.stream_rows
    assert np.diff(first).max() == p.max_words
    for u in range(len(first) - 1):
        rb, k = divmod(u, per_row)
        for lane in range(32):
            bits = "".join(f"{x:032b}"[::-1] for x in words[first[u]:first[u + 1], lane])
            at = 0
            for cg in range(4 * k, min(4 * k + 4, cols // 64)):
                for h in range(2):
                    for j in range(16):
                        n = 1
                        while bits[at:at + n] not in book:
                            n += 1
                        e = book[bits[at:at + n]]
                        at += n
                        four = int(sm[rb, cg, h, lane, j // 4])
                        out[16 * rb + 8 * h + lane // 4, 64 * cg + 16 * (lane % 4) + j] = \
                            (four >> sign[j % 4] & 1) << 15 | e << 7 | four >> mantissa[j % 4] & 0x7F
            assert "1" not in bits[at:] and len(bits) - at >= 0
    return out


@pytest.mark.parametrize("rows,cols", [(1, 1), (20, 300), (48, 130)])
def test_the_compressed_form_is_the_stated_one(rows, cols):
    w = _bf16((rows, cols), 0.05, rows)
    c = df11.compress_linear(w.cuda())
    got = _lane_streams(c)
    want = np.zeros(got.shape, np.uint16)
    want[:rows, :cols] = w.view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(got, want)


ROUND_TRIPS = ["gaussian", "one exponent", "mix", "every word", "long codes", "uneven rows"]


@pytest.mark.parametrize("kind", ROUND_TRIPS)
@pytest.mark.parametrize("rows,cols", [(16, 64), (1, 1), (33, 1000), (513, 4160), (300, 65)])
def test_round_trip(kind, rows, cols):
    n = rows * cols
    if kind == "gaussian":
        w = _bf16((n,), 0.02, 1)
    elif kind == "every word":
        w = torch.arange(n, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    elif kind == "long codes":      # lengths up to 32 bits, but for the limit
        w = workloads.fibonacci_exponents(seed=2)[:n].clone().view(torch.bfloat16)
    elif kind == "uneven rows":     # rows whose streams are far longer than others'
        w = torch.ones(n, dtype=torch.bfloat16)
        w[n // 2:] = workloads.gaussian_bf16(n - n // 2, 1.0, 4).view(torch.bfloat16)
    else:
        w = _words(kind, n)
    w = w.view(rows, cols)
    c = df11.compress_linear(w.cuda())
    err = df11.new_error_word()
    got = df11.decode_weight(c, err=err)
    torch.cuda.synchronize()
    df11.check_device_error(err)
    assert torch.equal(got.cpu().view(torch.int16), w.view(torch.int16))
    assert c.shape == (rows, cols) and c.params.max_words <= 32


@pytest.mark.parametrize("tokens", [1, 40])
def test_long_codes_in_the_product(tokens):
    w = workloads.fibonacci_exponents(seed=2)[:208 * 1280].clone().view(torch.bfloat16)
    w = w.view(208, 1280)
    w = torch.where(w.float().abs() < 1e15, w, torch.zeros_like(w))   # finite sums
    x = _bf16((tokens, 1280), 1.0, 2).cuda()
    y, = _run([df11.compress_linear(w.cuda())], [x], out_dtype=torch.float32)
    _check(w, x, y)


def test_sources_of_a_weight():
    w = _bf16((77, 150), 0.03, 1)
    ref = df11.compress_linear(w.cuda())
    for other in (w, w.cuda().view(torch.int16), w.cuda().t().contiguous().t(),
                  df11.compress(w), df11.compress_on_device(w.cuda()),
                  w.view(torch.int16).numpy()):
        c = df11.compress_linear(other)
        assert c.shape == (77, 150)
        assert torch.equal(c.streams, ref.streams) and torch.equal(c.table, ref.table)
        assert torch.equal(c.unit_rows, ref.unit_rows)
        assert torch.equal(c.sign_mantissa, ref.sign_mantissa)
    # kept in host memory and back
    x = _bf16((2, 150), 1.0, 5)
    y, = _run([ref.to("cpu").to("cuda")], [x.cuda()])
    _check(w, x, y)
    # a view that is not 16-byte aligned
    buf = torch.zeros(77 * 160 + 1, dtype=torch.bfloat16, device="cuda")
    odd = buf[1:1 + 77 * 150].view(77, 150)
    odd.copy_(w)
    assert torch.equal(df11.compress_linear(odd).streams, ref.streams)


def test_size_is_about_eleven_bits_per_weight():
    c = df11.compress_linear(_bf16((2048, 4096), 1 / 64, 3).cuda())
    bits = 8 * c.compressed_bytes() / (2048 * 4096)
    assert 10.5 < bits < 11.3, bits


@pytest.mark.parametrize("tokens", [4, 40])
@pytest.mark.parametrize("field", ["unit_rows", "table", "streams"])
def test_corrupt_weights_are_flagged_and_the_next_call_is_right(tokens, field):
    # rows of units out of order, an empty table, streams of the longest codewords: every
    # one is caught by a check of the kernel's own
    w = workloads.adversarial_mix(256 * 1024, seed=5).view(torch.bfloat16).view(256, 1024)
    c = df11.compress_linear(w.cuda())
    x = _bf16((tokens, 1024), 1.0, 2).cuda()
    good = c.table.clone(), c.unit_rows.clone(), c.streams.clone()
    if field == "unit_rows":
        c.unit_rows[5] = 1 << 28
    elif field == "table":
        c.table.zero_()                       # no codeword, of no length
    else:
        c.streams.fill_(-1)                   # the longest codeword, all along
    err = df11.new_error_word()
    df11.decode_linear([c], [x], err=err)
    torch.cuda.synchronize()
    with pytest.raises(df11.Df11Error):
        df11.check_device_error(err)
    c.table.copy_(good[0])
    c.unit_rows.copy_(good[1])
    c.streams.copy_(good[2])
    y, = _run([c], [x], out_dtype=torch.float32)
    _check(w, x, y)


@pytest.mark.parametrize("tokens", [1, 32, 40, 300])
def test_long_sums_do_not_drift(tokens):
    # the sum of 12288 positive products has a relative error of the order of fp32's own
    # rounding, not of 12288 times it.  Exact products; a tile (64 columns, 16 products a step)
    # or 512 columns are summed where each of at most 32 additions may cut off one unit
    # (2^-23) of a partial sum of a part, the parts then with half a unit each: at most
    # 32 2^-23 (the parts' own) + 200 2^-24 relative, and in the mean far less
    cols = 12288
    w = _bf16((64, cols), 0.02, 1).abs()
    x = _bf16((tokens, cols), 1.0, 2).abs().cuda()
    y, = _run([df11.compress_linear(w.cuda())], [x], out_dtype=torch.float32)
    want = x.cpu().double() @ w.double().T
    rel = ((y.cpu().double() - want) / want).abs()
    assert float(rel.max()) <= 32 * 2.0 ** -23 + 200 * 2.0 ** -24


@pytest.mark.parametrize("tokens", [2, 50])
def test_activations_of_special_values(tokens):
    # a weight of one: the products are x itself
    w = torch.zeros(16, 64, dtype=torch.bfloat16)
    w[0, 0] = 1.0
    d = df11.compress_linear(w.cuda())
    x = torch.zeros(tokens, 64, dtype=torch.bfloat16)
    x[1, 0] = float("nan")
    for v in (-3e38, -200.0, 200.0, 3e38):
        x[0, 0] = v
        for act, want in (("relu", max(v, 0.0)), ("gelu", max(v, 0.0)), ("gelu_tanh", max(v, 0.0)),
                          ("silu", max(v, 0.0))):
            y, = _run([d], [x.cuda()], activations=[act], out_dtype=torch.float32)
            got = float(y[0, 0])
            assert got == float(torch.tensor(want).to(torch.bfloat16)), (act, v, got)
            assert torch.isnan(y[1, 0]), act


def test_streams_by_object_and_handle_and_dropped_plans():
    w = _bf16((512, 768), 0.05, 1)
    side = torch.cuda.Stream()
    wc, x = w.cuda(), _bf16((5, 768), 1.0, 2).cuda()
    torch.cuda.synchronize()
    c = df11.compress_linear(wc, stream=side)
    for stream in (side, side.cuda_stream, 0, None):
        ys = [torch.empty(5, 512, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        for y in ys:      # a plan of its own for each, dropped while it may still run
            df11.LinearPlan([c], [x], [y]).run(stream=stream)
            torch.empty(1 << 20, device="cuda").fill_(float("nan"))
        torch.cuda.synchronize()
        for y in ys:
            _check(w, x, y)


def test_words_as_activations_and_other_word_types():
    w = _bf16((64, 128), 0.1, 1)
    x = _bf16((3, 128), 1.0, 2).cuda()
    c = df11.compress_linear(w.cuda().view(torch.uint16))
    y, = _run([c], [x.view(torch.int16)], out_dtype=torch.float32)
    _check(w, x, y)


@pytest.mark.parametrize("tokens", [3, 40])
def test_a_weight_of_more_than_two_to_the_31_elements(tokens):
    rows, cols = 45000, 49152
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, 5000):
        w[i:i + 5000] = torch.randn(5000, cols, generator=g, device="cuda").mul_(cols ** -0.5)
    c = df11.compress_linear(w)
    x = _bf16((tokens, cols), 1.0, 2).cuda()
    y, = _run([c], [x], out_dtype=torch.float32)
    pick = torch.cat([torch.arange(40), torch.arange(21800, 21860), torch.arange(rows - 40, rows)])
    _check(w[pick.cuda()], x, y[:, pick.cuda()])
    assert torch.isfinite(y).all()
    del w, c
    torch.cuda.empty_cache()


def test_bf16_outputs_of_long_rows():
    # beyond 65536 columns BF16 outputs too are summed in parts of 512 columns (a part's own
    # error at most 32 2^-23, the parts' 160 additions half a unit each), then rounded once
    cols = 80000
    w = _bf16((48, cols), 0.02, 1).abs()
    x = _bf16((40, cols), 1.0, 2).abs().cuda()
    y, = _run([df11.compress_linear(w.cuda())], [x])
    want = x.cpu().double() @ w.double().T
    rel = ((y.cpu().double() - want) / want).abs()
    assert float(rel.max()) <= 2.0 ** -8 + 32 * 2.0 ** -23 + 160 * 2.0 ** -24


@pytest.mark.parametrize("rows,cols,tokens", [(4096, 4096, 40), (4096, 12288, 128), (500, 8192, 130),
                                              (1013, 1411, 77), (96, 5000, 33), (2064, 2048, 260),
                                              (16, 12288, 1100), (7000, 640, 50)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_tiles_that_thread_blocks_share(rows, cols, tokens, out):
    w = _bf16((rows, cols), cols ** -0.5, 1)
    x = _bf16((tokens, cols), 1.0, 2).cuda()
    bias = _bf16((rows,), 1.0, 3)
    mul, res = _bf16((tokens, rows), 1.0, 4), _bf16((tokens, rows), 1.0, 5)
    d = df11.compress_linear(w.cuda())
    kw = dict(biases=[bias.cuda()], multipliers=[mul.cuda()], residuals=[res.cuda()], out_dtype=out)
    y, = _run([d], [x], **kw)
    again, = _run([d], [x], **kw)
    assert torch.equal(y.view(torch.uint8), again.view(torch.uint8))
    _check(w, x, y, bias=bias, multiplier=mul, residual=res)
