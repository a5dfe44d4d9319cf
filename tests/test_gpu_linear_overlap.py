"""Outputs on the memory of their own operands, through the binding."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu

df11 = pytest.importorskip("huffman_decode_df11_b200")


@pytest.mark.parametrize("tokens", [1, 4, 40])
def test_outputs_on_their_own_operands_are_refused_and_beside_them_right(tokens):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    w = workloads.gaussian_bf16(128 * 128, 0.1, 1).view(torch.bfloat16).view(128, 128).cuda()
    d = df11.compress_linear(w)
    both = workloads.gaussian_bf16(tokens * 256, 1.0, 2).view(torch.bfloat16).view(tokens, 256).cuda()
    x, y = both[:, :128], both[:, 128:]
    want, = df11.decode_linear([d], [x.clone()], multipliers=[y.clone()])
    with pytest.raises(ValueError, match="shares memory"):
        df11.LinearPlan([d], [x], [x])
    with pytest.raises(ValueError, match="shares memory"):
        df11.decode_linear([d], [x], [both[:, 64:192]])
    with pytest.raises(ValueError, match="shares memory"):
        df11.decode_linear([d], [x], [y], residuals=[both[:, 100:228]])
    assert df11.decode_linear([d], [x], [y], multipliers=[y])[0] is y  # in place, columns of one buffer
    torch.cuda.synchronize()
    assert torch.equal(y, want)
