"""The embedding on a compressed table against the formula on the original one.

Lookup: with scale 1 and BF16 out, the same bits; fp32 out the same values.
Scaled: one fp32 product (2^-24 relative), rounded once to BF16 (2^-8 relative) or
not at all.

Gradient: a row with k tokens is a sum of k terms in fp32, in any order within
k - 1 additions and one scaling, so with S = |scale| sum |g|,
    e = (k + 1) 2^-24 S        (2^-24: half a unit, additions round to nearest)
and one rounding to the result's type (BF16 2^-8, fp32 in the (k + 1) already); an
addition to what is there is one more fp32 term.
"""
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


def _table(rows, dim, seed=1, std=0.02):
    return workloads.gaussian_bf16(rows * dim, std, seed).view(torch.bfloat16).view(rows, dim)


def _ids(n, rows, seed, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, rows, (n,), generator=g).to(dtype)


def _lookup(d, ids, **kw):
    err = df11.new_error_word()
    out = df11.decode_embedding(d, ids.cuda(), err=err, **kw)
    torch.cuda.synchronize()
    df11.check_device_error(err)
    return out.cpu()


def _bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("rows,dim,n", [
    (1, 1, 1), (40, 16, 7), (1000, 4096, 5), (1000, 4096, 300), (5003, 333, 1000), (77, 1003, 64),
    (3, 40000, 9), (20000, 64, 5000), (400, 2304, 33), (700, 8192, 65), (9, 17, 400)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_rows_come_back_bit_for_bit(rows, dim, n, dtype):
    w = _table(rows, dim, rows + dim)
    ids = _ids(n, rows, n, dtype)
    ids[0] = rows - 1
    ids[-1] = 0
    d = df11.compress_on_device(w.cuda())
    assert torch.equal(_bits(_lookup(d, ids)), _bits(w[ids.long()]))
    got = _lookup(d, ids, out_dtype=torch.float32)
    assert torch.equal(got, w[ids.long()].float())


def test_every_row_of_a_table():
    w = _table(3000, 500)
    d = df11.compress_on_device(w.cuda())
    assert torch.equal(_bits(_lookup(d, torch.arange(3000))), _bits(w))


@pytest.mark.parametrize("chunk_bytes", [8, 16, 24])
def test_chunk_sizes_and_the_host_builder(chunk_bytes):
    w = _table(600, 1040)
    d = df11.to_device(df11.compress(w, chunk_bytes))
    ids = _ids(200, 600, 3)
    assert torch.equal(_bits(_lookup(d, ids)), _bits(w[ids]))


@pytest.mark.parametrize("kind", ["one exponent", "mix", "every word", "drift", "long codes"])
def test_other_exponent_distributions(kind):
    rows, dim = 512, 1000
    n = rows * dim
    if kind == "one exponent":
        g = torch.Generator().manual_seed(1)
        w = torch.where(torch.rand(n, generator=g) < 0.5, 1.0, -1.5).to(torch.bfloat16)
    elif kind == "mix":
        w = workloads.adversarial_mix(n, seed=5).view(torch.bfloat16)
    elif kind == "every word":
        w = torch.arange(n, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    elif kind == "long codes":
        w = workloads.fibonacci_exponents(seed=2)[:n].clone().view(torch.bfloat16)
    else:  # rows whose codes are short, then long: the positions are far from even
        w = torch.ones(n, dtype=torch.bfloat16)
        w[n // 2:] = workloads.gaussian_bf16(n - n // 2, 1.0, 4).view(torch.bfloat16)
    w = w.view(rows, dim)
    d = df11.compress_on_device(w.cuda())
    ids = torch.cat([torch.arange(rows), _ids(500, rows, 1)])
    assert torch.equal(_bits(_lookup(d, ids)), _bits(w[ids]))


@pytest.mark.parametrize("scale", [64.0, 0.3, -1.0, 0.0])
@pytest.mark.parametrize("dim", [128, 131])
def test_scaled(scale, dim):
    w = _table(300, dim)
    ids = _ids(100, 300, 2)
    d = df11.compress_on_device(w.cuda())
    want = w[ids].double() * float(np.float32(scale))
    got = _lookup(d, ids, scale=scale, out_dtype=torch.float32).double()
    assert torch.all((got - want).abs() <= 2.0 ** -24 * want.abs())
    got = _lookup(d, ids, scale=scale).double()
    assert torch.all((got - want).abs() <= (2.0 ** -8 + 2.0 ** -23) * want.abs())


@pytest.mark.parametrize("dim", [256, 99])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_shapes_strides_and_bytes_around_the_rows(dim, dtype):
    w = _table(200, dim)
    d = df11.compress_on_device(w.cuda())
    ids = _ids(24, 200, 6)
    assert _lookup(d, ids.view(2, 3, 4), out_dtype=dtype).shape == (2, 3, 4, dim)
    buf = torch.full((26, dim + 5), 3.0, dtype=dtype, device="cuda")
    out = buf[1:25, 2:dim + 2]
    df11.decode_embedding(d, ids.cuda(), out=out)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), w[ids].to(dtype))
    out.fill_(3.0)
    assert torch.all(buf == 3.0)


def test_ids_outside_the_table_give_zeros_and_an_error():
    w = _table(50, 300)
    d = df11.compress_on_device(w.cuda())
    for dtype, far in ((torch.int32, 2 ** 31 - 1), (torch.int64, 2 ** 40)):
        ids = torch.tensor([3, -1, 50, 49, far, 7], dtype=dtype)
        err = df11.new_error_word()
        out = df11.decode_embedding(d, ids.cuda(), err=err)
        torch.cuda.synchronize()
        with pytest.raises(df11.Df11Error, match="INDEX"):
            df11.check_device_error(err)
        out = out.cpu()
        assert torch.equal(_bits(out[[0, 3, 5]]), _bits(w[[3, 49, 7]]))
        assert torch.count_nonzero(out[[1, 2, 4]]) == 0


def test_no_tokens():
    d = df11.compress_on_device(_table(50, 30).cuda())
    assert df11.decode_embedding(d, torch.zeros(0, dtype=torch.int64, device="cuda")).shape == (0, 30)


def test_corrupt_counts_are_flagged_and_the_next_lookup_is_right():
    w = _table(500, 1024)
    d = df11.compress_on_device(w.cuda())
    ids = torch.arange(500)
    good = int(d.chunk_counts[300])
    d.chunk_counts[300] = good + 1
    err = df11.new_error_word()
    df11.decode_embedding(d, ids.cuda(), err=err)
    torch.cuda.synchronize()
    with pytest.raises(df11.Df11Error):
        df11.check_device_error(err)
    d.chunk_counts[300] = good
    assert torch.equal(_bits(_lookup(d, ids)), _bits(w))


def test_plan_in_a_captured_graph_reads_the_ids_of_the_replay():
    w = _table(3000, 640)
    d = df11.compress_on_device(w.cuda())
    ids = torch.zeros(70, dtype=torch.int32, device="cuda")
    out = torch.empty(70, 640, dtype=torch.bfloat16, device="cuda")
    plan = df11.EmbeddingPlan(d, ids, out)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        plan.run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            plan.run()
        for seed in range(3):
            want = _ids(70, 3000, seed, torch.int32)
            ids.copy_(want)
            g.replay()
            side.synchronize()
            assert torch.equal(_bits(out.cpu()), _bits(w[want.long()]))


def test_a_table_of_nearly_two_to_the_32_elements():
    rows, dim = 65500, 65500
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, 5000):
        n = min(5000, rows - i)
        w[i:i + n] = torch.randn(n, dim, generator=g, device="cuda").mul_(0.02)
    d = df11.compress_on_device(w)
    ids = torch.cat([torch.arange(3), torch.arange(32700, 32860), torch.arange(rows - 9, rows)])
    want = w[ids.cuda()].cpu()
    del w
    got = _lookup(d, ids)
    assert torch.equal(_bits(got), _bits(want))
    del d
    torch.cuda.empty_cache()


def test_streams_by_object_and_handle():
    w = _table(300, 256)
    d = df11.compress_on_device(w.cuda())
    ids = _ids(64, 300, 1)
    dev_ids, grad = ids.cuda(), torch.randn(64, 256, generator=torch.Generator().manual_seed(1)).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, 0, None):
        out = df11.decode_embedding(d, dev_ids, stream=stream)
        dw = df11.embedding_gradient(dev_ids, grad, 300, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(_bits(out.cpu()), _bits(w[ids]))
        _check_gradient(ids, grad, 300, dw)


# ---- gradient -----------------------------------------------------------------


def _check_gradient(ids, grad, rows, got, scale=1.0, before=None):
    ids, g = ids.cpu().long().reshape(-1), grad.detach().cpu().double()
    g = g.reshape(len(ids), -1)
    s = float(np.float32(scale))
    ok = (ids >= 0) & (ids < rows)
    want = torch.zeros(rows, g.shape[1], dtype=torch.float64).index_add_(0, ids[ok], g[ok]) * s
    S = torch.zeros_like(want).index_add_(0, ids[ok], g[ok].abs()) * abs(s)
    k = torch.bincount(ids[ok], minlength=rows).double()[:, None]
    if before is not None:
        b = before.cpu().double()
        want, S, k = want + b, S + b.abs(), k + 1
        untouched = (k == 1).squeeze(1)
        assert torch.equal(got.cpu()[untouched], before.cpu()[untouched])
    e = (k + 1) * 2.0 ** -24 * S
    if got.dtype == torch.bfloat16:
        e = e + 2.0 ** -8 * (want.abs() + e)
    err = (got.detach().cpu().double() - want).abs()
    assert torch.all(err <= e + 1e-40), float((err - e).max())


def _gradient(ids, grad, rows, **kw):
    err = df11.new_error_word()
    out = df11.embedding_gradient(ids.cuda(), grad, rows, err=err, **kw)
    torch.cuda.synchronize()
    df11.check_device_error(err)
    return out


GRADS = [(70000, 152000, 8), (2000, 511, 40), (2000, 512, 40), (1025, 262143, 4), (1, 1, 1), (1000, 1, 1), (300, 5003, 333), (8192, 200, 64), (4096, 50000, 40),
         (5000, 3, 130), (33, 1000, 4096), (20000, 151936, 16), (64, 64, 8192), (9000, 300, 24)]


@pytest.mark.parametrize("n,rows,dim", GRADS)
@pytest.mark.parametrize("gtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("otype", [torch.float32, torch.bfloat16])
def test_gradient(n, rows, dim, gtype, otype):
    ids = _ids(n, rows, n + rows, torch.int32 if n % 2 else torch.int64)
    g = torch.Generator().manual_seed(n)
    grad = torch.randn(n, dim, generator=g).to(gtype).cuda()
    out = _gradient(ids, grad, rows, out_dtype=otype, scale=3.7)
    _check_gradient(ids, grad, rows, out, 3.7)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 4095, 4097, 33000])
@pytest.mark.parametrize("dim", [16, 17])
def test_one_token_shared_by_all_and_by_half(n, dim):
    grad = torch.randn(n, dim, generator=torch.Generator().manual_seed(1)).cuda()
    for ids in (torch.full((n,), 5), torch.where(torch.arange(n) % 2 == 0, 5, torch.arange(n) % 90)):
        _check_gradient(ids, grad, 91, _gradient(ids, grad, 91))


@pytest.mark.parametrize("otype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim", [128, 77])
def test_accumulate_touches_only_rows_with_tokens(otype, dim):
    ids = _ids(500, 400, 3)
    grad = torch.randn(500, dim, generator=torch.Generator().manual_seed(2)).cuda()
    before = torch.randn(400, dim, generator=torch.Generator().manual_seed(3)).to(otype)
    out = before.clone().cuda()
    got = _gradient(ids, grad, 400, out=out, accumulate=True, scale=0.5)
    assert got is out
    _check_gradient(ids, grad, 400, out, 0.5, before)


@pytest.mark.parametrize("dim", [64, 65])
def test_gradient_strides_and_bytes_around_the_rows(dim):
    n, rows = 300, 120
    ids = _ids(n, rows, 8)
    gb = torch.randn(n, dim + 3, generator=torch.Generator().manual_seed(2)).cuda()
    grad = gb[:, 1:dim + 1]
    buf = torch.full((rows + 2, dim + 7), 9.0, device="cuda")
    out = buf[1:rows + 1, 3:dim + 3]
    _gradient(ids, grad, rows, out=out)
    _check_gradient(ids, grad, rows, out)
    out.fill_(9.0)
    assert torch.all(buf == 9.0)


def test_gradient_of_ids_outside_the_table():
    ids = torch.tensor([2, -1, 9, 2, 10, 2 ** 40, 0], dtype=torch.int64)
    grad = torch.randn(7, 48, generator=torch.Generator().manual_seed(2)).cuda()
    err = df11.new_error_word()
    out = df11.embedding_gradient(ids.cuda(), grad, 10, err=err)
    torch.cuda.synchronize()
    with pytest.raises(df11.Df11Error, match="INDEX"):
        df11.check_device_error(err)
    _check_gradient(ids, grad, 10, out)


def test_no_tokens_give_a_zero_gradient():
    ids = torch.zeros(0, dtype=torch.int64)
    out = torch.full((70, 48), 5.0, device="cuda")
    _gradient(ids, torch.zeros(0, 48, device="cuda"), 70, out=out)
    assert torch.count_nonzero(out) == 0
    out.fill_(5.0)
    _gradient(ids, torch.zeros(0, 48, device="cuda"), 70, out=out, accumulate=True)
    assert torch.all(out == 5.0)


def test_a_gradient_repeats_bit_for_bit():
    ids = _ids(20000, 500, 4)
    ids[::3] = 17
    grad = torch.randn(20000, 256, generator=torch.Generator().manual_seed(2)).cuda()
    first = _gradient(ids, grad, 500)
    for _ in range(5):
        assert torch.equal(_gradient(ids, grad, 500), first)


def test_gradient_against_differences():
    # f(W) = sum over tokens of <c_t, s W[ids_t]> is linear in W: its difference in one
    # entry is exact up to the lookup's rounding
    rows, dim, s = 12, 32, 2.0
    w = _table(rows, dim, std=1.0)
    ids = _ids(40, rows, 5)
    c = torch.randint(-4, 5, (40, dim), generator=torch.Generator().manual_seed(1)).float()
    dw = _gradient(ids, c.cuda(), rows, scale=s).cpu()
    for v, j in ((0, 0), (3, 31), (11, 7), (int(ids[0]), 5)):
        up = w.clone()
        up[v, j] = 2.0
        down = w.clone()
        down[v, j] = -2.0
        f = [float((_lookup(df11.compress_on_device(t.cuda()), ids, scale=s,
                            out_dtype=torch.float32).double() * c.double()).sum())
             for t in (up, down)]
        assert abs((f[0] - f[1]) / 4.0 - float(dw[v, j])) < 1e-9


def test_gradient_in_captured_graphs():
    rows, n, dim = 300, 200, 64
    ids = torch.zeros(n, dtype=torch.int64, device="cuda")
    grad = torch.zeros(n, dim, device="cuda")
    outs = [torch.empty(rows, dim, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        df11.embedding_gradient(ids, grad, rows, out=outs[0])
        graphs = []
        for o in outs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                df11.embedding_gradient(ids, grad, rows, out=o)
            graphs.append(g)
        for seed in range(4):
            i = _ids(n, rows, seed)
            x = torch.randn(n, dim, generator=torch.Generator().manual_seed(seed))
            ids.copy_(i)
            grad.copy_(x)
            graphs[seed % 2].replay()
            side.synchronize()
            _check_gradient(i, x, rows, outs[seed % 2])


def test_lookup_linear_and_gradient_together():
    """A step of a model's ends: embed, project, and the table's gradient from the
    projection's output, then the updated table compressed again and looked up."""
    rows, dim, out_dim = 400, 256, 320
    table, w = _table(rows, dim, 2), _table(out_dim, dim, 3, std=0.05)
    d, dl = df11.compress_on_device(table.cuda()), df11.compress_linear(w.cuda())
    ids = _ids(90, rows, 9).view(6, 15).cuda()
    h = df11.decode_embedding(d, ids, scale=16.0)
    y, = df11.decode_linear([dl], [h.view(90, dim)], out_dtype=torch.float32)
    torch.cuda.synchronize()
    want = (table[ids.cpu()].double() * 16).view(90, dim) @ w.double().T
    S = (table[ids.cpu()].double().abs() * 16).view(90, dim) @ w.double().abs().T
    # the lookup is exact here (a power of two); the product as in its own tests
    assert torch.all((y.cpu().double() - want).abs() <= (dim + 16) * 2.0 ** -23 * S)
    gh = (y @ w.float().cuda()).view(6, 15, dim)
    dw = _gradient(ids, gh, rows, scale=16.0)
    _check_gradient(ids, gh, rows, dw, 16.0)
    updated = (table.float().cuda() - 1e-3 * dw).to(torch.bfloat16)
    d2 = df11.compress_on_device(updated)
    assert torch.equal(_bits(_lookup(d2, torch.arange(rows))), _bits(updated.cpu()))


@pytest.mark.parametrize("rows,dim,tokens", [(20011, 1000, 9000), (3, 16384, 100), (40000, 136, 1)])
def test_rows_without_tokens_are_zero_in_every_part(rows, dim, tokens):
    # the table's first and last rows are set to zero beside different steps: ids in all parts,
    # and gaps between output rows that stay as they were
    ids = _ids(tokens, rows, 5)
    ids[0], ids[-1] = rows - 1, 0
    grad = torch.randn(tokens, dim, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    wide = torch.full((rows, dim + 8), 7.0, device="cuda")
    df11.embedding_gradient(ids.cuda(), grad, rows, out=wide[:, :dim])
    _check_gradient(ids, grad, rows, wide[:, :dim])
    assert bool((wide[:, dim:] == 7.0).all())
    full = torch.full((rows, dim), 7.0, device="cuda")
    df11.embedding_gradient(ids.cuda(), grad, rows, out=full)
    assert torch.equal(full, wide[:, :dim])


def test_gradient_rows_that_end_inside_a_tile():
    # BF16 and fp32 rows of which the last column tile has 8 columns, in pieces of every size
    for tokens in (1, 7, 8, 9, 33, 600):
        for dtype in (torch.bfloat16, torch.float32):
            ids = _ids(tokens, 37, tokens)
            grad = torch.randn(tokens, 1032, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
            dw = df11.embedding_gradient(ids.cuda(), grad, 37)
            _check_gradient(ids, grad, 37, dw)


@pytest.mark.parametrize("scale", [64.0, -1.5, 2.0 ** -60, 2.0 ** 60, 1.0078125, 0.1])
def test_scaled_words_of_every_kind(scale):
    # every BF16 word, infinities, NaN and subnormal ones among them: the product in 64 bits,
    # rounded once (half a unit of the smallest subnormal, 2^-134, where that is all there is)
    w = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).reshape(256, 256)
    d = df11.compress_on_device(w.cuda())
    ids = torch.arange(256)
    got = _lookup(d, ids, scale=scale)
    want = w.double() * float(np.float32(scale))
    nan = want.isnan()
    assert torch.equal(got.cpu().isnan(), nan)
    near = want.float().to(torch.bfloat16)  # exact in fp32 for two factors of 8 bits
    tiny = want.abs() < 2.0 ** -126
    if scale != 0.1:
        same = ~nan & ~tiny
        assert torch.equal(got.cpu()[same], near[same])
    else:
        fin = ~nan & ~tiny & (want.abs() < 3e38)
        err = (got.cpu().double() - want).abs()[fin]
        assert torch.all(err <= 2.0 ** -8 * want.abs()[fin] * (1 + 2.0 ** -15))
    assert torch.all((got.cpu().double() - want).abs()[tiny] <= 2.0 ** -134 * (1 + 2.0 ** -8))


@pytest.mark.parametrize("chunk_bytes", [8, 16, 24])
@pytest.mark.parametrize("dim", [1, 5, 48, 64, 100, 160, 256, 371, 512, 1003, 1024])
def test_many_short_rows(dim, chunk_bytes):
    # more rows than the device holds warps: a few lanes each
    rows = 40000 // dim + 3
    w = _table(rows, dim)
    d = df11.compress_on_device(w.cuda(), chunk_bytes=chunk_bytes)
    ids = _ids(9001, rows, 1)
    ids[:3], ids[-3:] = rows - 1, 0
    assert torch.equal(_bits(_lookup(d, ids)), _bits(w[ids]))
    got = _lookup(d, ids.to(torch.int32), scale=0.3, out_dtype=torch.float32).cpu()
    assert torch.equal(got, w[ids].float() * float(np.float32(0.3)))
    wide = torch.full((9001, dim + 3), 5.0, dtype=torch.bfloat16, device="cuda")
    df11.decode_embedding(d, ids.cuda(), out=wide[:, :dim])
    assert torch.equal(_bits(wide[:, :dim].cpu()), _bits(w[ids])) and bool((wide[:, dim:] == 5).all())
    ids[100], ids[8000] = -1, rows
    err = df11.new_error_word()
    got = df11.decode_embedding(d, ids.cuda(), err=err).cpu()
    want = w[ids.clamp(0, rows - 1)].clone()
    want[100], want[8000] = 0, 0
    assert torch.equal(_bits(got), _bits(want))
    with pytest.raises(Exception):
        df11.check_device_error(err)


def test_many_short_rows_of_long_codes():
    # words whose codes differ most in length, and blocks far from the proportional guess
    g = torch.Generator().manual_seed(3)
    easy = torch.full((30000, 24), 1.0, dtype=torch.bfloat16)
    hard = torch.randint(-32768, 32767, (6000, 24), generator=g, dtype=torch.int32).to(torch.int16)
    w = torch.cat([easy, hard.view(torch.bfloat16), easy[:500]])
    d = df11.compress_on_device(w.cuda())
    ids = torch.cat([torch.arange(29000, 36500), _ids(3000, len(w), 2)])
    assert torch.equal(_bits(_lookup(d, ids)), _bits(w[ids]))
