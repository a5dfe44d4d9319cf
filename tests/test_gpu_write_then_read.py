"""What the library writes on the device may be read by its very next launch in the stream,
although launches begin to read before the previous kernel is done."""
import ctypes

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


def _words(rows, cols):
    return workloads.gaussian_bf16(rows * cols, 0.05, 1).view(torch.bfloat16).view(rows, cols).cuda()


def test_a_decode_table_and_the_lookup_and_decode_behind_it():
    w = _words(500, 640)
    d = df11.compress_on_device(w)
    ids = torch.arange(0, 500, 7, device="cuda")
    out, whole = w[ids].clone(), w.clone().view(-1)
    lookup, decode = df11.EmbeddingPlan(d, ids, out), df11.DecodePlan([d], [whole])
    L, stream = df11.lib(), torch.cuda.current_stream().cuda_stream
    for plan, got, want in [(lookup, out, w[ids]), (decode, whole, w.view(-1))] * 10:
        d.decode_table.fill_(255)
        got.zero_()
        torch.cuda.synchronize()
        assert L.df11_build_decode_table(d._ptr("luts"), d._ptr("code_lengths"), d.params.num_luts,
                                         d.decode_table.data_ptr(), stream) == 0
        plan.run()
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_a_compressed_weight_and_the_product_and_decoding_behind_it():
    w = _words(64, 1024)
    c = df11.compress_linear(w)
    x = _words(3, 1024)
    want, = df11.decode_linear([c], [x], out_dtype=torch.float32)
    y, tiles = torch.empty_like(want), torch.empty(64 * 1024, dtype=torch.bfloat16, device="cuda")
    plan, desc = df11.LinearPlan([c], [x], [y]), c.desc()
    plan.run()
    L, stream = df11.lib(), torch.cuda.current_stream().cuda_stream
    for i in range(20):
        c.streams.fill_(0)
        c.sign_mantissa.fill_(0)
        torch.cuda.synchronize()
        assert L.df11_linear_weight_finish(w.data_ptr(), ctypes.byref(desc), stream) == 0
        if i % 2:
            plan.run()
            torch.cuda.synchronize()
            assert torch.equal(y, want)
        else:
            assert L.df11_linear_unpack(ctypes.byref(desc), tiles.data_ptr(), None, stream) == 0
            torch.cuda.synchronize()
            got = tiles.view(4, 16, 16, 64).permute(0, 2, 1, 3).reshape(64, 1024)
            assert torch.equal(got.view(torch.int16), w.view(torch.int16))
