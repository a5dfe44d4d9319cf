"""A weight whose words change between the two calls of the builder: wrong, but nothing is
written outside of its buffers."""
import ctypes

import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu

df11 = pytest.importorskip("huffman_decode_df11_b200")


@pytest.mark.parametrize("rows,cols", [(16, 64), (48, 1000), (300, 4160)])
def test_nothing_behind_the_streams_is_written(rows, cols):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    w = torch.ones(rows, cols, dtype=torch.bfloat16)
    w[0, :8] = workloads.gaussian_bf16(8, 1e-3, 1).view(torch.bfloat16)     # ones are one bit each
    w = w.cuda()
    c = df11.compress_linear(w)
    n, guard = c.streams.numel(), 1 << 16
    room = torch.full((n + guard,), -559038737, dtype=torch.int32, device="cuda")
    d = c.desc()
    d.streams = room.data_ptr()
    other = w[0, :8].repeat(rows, -(-cols // 8))[:, :cols].contiguous()     # the longest codewords
    assert df11.lib().df11_linear_weight_finish(other.data_ptr(), ctypes.byref(d), None) == 0
    torch.cuda.synchronize()
    assert torch.all(room[n:] == -559038737) and not torch.all(room[:n] == -559038737)
    # the words that were counted give the weight again
    assert df11.lib().df11_linear_weight_finish(w.data_ptr(), ctypes.byref(d), None) == 0
    torch.cuda.synchronize()
    assert torch.equal(room[:n], c.streams)
