"""The linear product on whole numbers, whose sums are exact in fp32 in any order: every output
has to be the very number, whatever the length, so that a lost or misplaced group of columns shows
(the general bound, which counts an error for every column, has room for one beyond 10000)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

df11 = pytest.importorskip("huffman_decode_df11_b200")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.init()


def _whole(shape, seed, limit=7):
    """Whole numbers from -limit to limit in BF16: sums of 2^24 / limit^2 products are exact."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-limit, limit + 1, shape, generator=g, device="cuda",
                         dtype=torch.int8).to(torch.bfloat16)


def _check(w, d, x, outs=(torch.float32, torch.bfloat16), **extras):
    want = torch.cat([x.float() @ w[i:i + 4096].float().t() for i in range(0, w.shape[0], 4096)], dim=1)
    if extras:
        want = (want + extras["bias"].float()).clamp(min=0) * extras["multiplier"].float()
        want += extras["residual"].float()
    assert float(want.abs().max()) < 2 ** 24
    kw = {} if not extras else dict(biases=[extras["bias"]], activations=["relu"],
                                    multipliers=[extras["multiplier"]], residuals=[extras["residual"]])
    for out in outs:
        err = df11.new_error_word()
        y, = df11.decode_linear([d], [x], out_dtype=out, err=err, **kw)
        torch.cuda.synchronize()
        df11.check_device_error(err)
        assert torch.equal(y, want.to(out))


LONG = [(512, 12288, 17), (40, 20000, 3), (16, 40000, 20), (5000, 12288, 40), (300, 80000, 50),
        (4099, 20000, 200), (7, 65537, 1), (2048, 12288, 8), (1000, 16384, 32), (33, 300000, 33)]


@pytest.mark.parametrize("rows,cols,tokens", LONG)
def test_long_rows(rows, cols, tokens):
    w, x = _whole((rows, cols), rows), _whole((tokens, cols), tokens)
    _check(w, df11.compress_linear(w), x)


@pytest.mark.parametrize("rows", [320, 333, 4096, 4100])
@pytest.mark.parametrize("cols", [512, 640, 1411, 4096])
@pytest.mark.parametrize("tokens", [1, 9, 24, 40, 128, 129, 700])
@pytest.mark.parametrize("extras", [torch.float32, torch.bfloat16])
def test_the_whole_epilogue(rows, cols, tokens, extras):
    w, x = _whole((rows, cols), 1), _whole((tokens, cols), 2)
    b, m, r = (_whole(s, i, 3).to(extras) for i, s in enumerate(((rows,), (tokens, rows), (tokens, rows))))
    _check(w, df11.compress_linear(w), x, bias=b, multiplier=m, residual=r)


@pytest.mark.parametrize("tokens", [3, 20, 40, 300])
def test_a_weight_of_more_than_two_to_the_31_elements(tokens):
    w = _whole((45000, 49152), 1)
    _check(w, df11.compress_linear(w), _whole((tokens, 49152), 2), outs=(torch.float32,))
    torch.cuda.empty_cache()


@pytest.mark.parametrize("counts", [(1, 33, 300), (40, 2, 7, 128), (1, 2, 3), (33, 0, 8, 9)])
def test_token_counts_of_both_paths_in_one_call(counts):
    w = _whole((272, 1411), 1)
    ds = [df11.compress_linear(w)] * len(counts)
    xs = [_whole((t, 1411), t) for t in counts]
    for out in (torch.float32, torch.bfloat16):
        ys = df11.decode_linear(ds, xs, out_dtype=out)
        for x, y in zip(xs, ys):
            assert torch.equal(y, (x.float() @ w.float().t()).to(out))


@pytest.mark.parametrize("tokens", [5, 40, 300])
@pytest.mark.parametrize("cols", [448, 1024])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_operands_off_their_16_byte_boundaries_one_at_a_time(tokens, cols, kind):
    rows = 304
    w, x = _whole((rows, cols), 1), _whole((tokens, cols), 2)
    d = df11.compress_linear(w)

    def place(t, off):  # the same values `off` elements into a buffer with 16-byte rows
        wide = torch.zeros(t.shape[0], t.shape[1] + 16, dtype=t.dtype, device="cuda")
        view = wide[:, off:off + t.shape[1]]
        view.copy_(t)
        return view

    b, m, r = (_whole(s, i, 3).to(kind) for i, s in enumerate(((1, rows), (tokens, rows), (tokens, rows))))
    want = ((x.float() @ w.float().t() + b.float()).clamp(min=0) * m.float() + r.float()).to(kind)
    for shifted in (None, "x", "y", "bias", "multiplier", "residual"):
        def at(name, t):
            return place(t, 3 if name == shifted else 0)
        y = at("y", torch.zeros_like(want))
        df11.decode_linear([d], [at("x", x)], [y], biases=[at("bias", b)[0]], activations=["relu"],
                           multipliers=[at("multiplier", m)], residuals=[at("residual", r)])
        assert torch.equal(y, want), shifted
