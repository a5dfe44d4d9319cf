"""The sums of the linear product where rounding alone does not hide them.

Products of BF16 are exact in fp32.  Beyond 32 tokens the columns are summed in parts of at
most 512: a part is a chain of at most 32 tensor-core additions (16 columns each), which may cut
off one unit (2^-23 relative) each, and the parts are added in fp32 with half a unit each.  So
for positive terms with the sum P
    |sum - P| <= (32 2^-23 + parts 2^-24) P.
"""
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


def _positive(shape, std, seed):
    n = shape[0] * shape[1]
    return workloads.gaussian_bf16(n, std, seed).view(torch.bfloat16).view(shape).abs().cuda()


@pytest.mark.parametrize("rows,cols,tokens", [(4096, 12288, 300), (4096, 65536, 300),
                                              (333, 12288, 70), (12288, 4096, 129)])
def test_a_residual_that_cancels_the_sum_leaves_its_error(rows, cols, tokens):
    # residual = -P rounded to fp32 (half a unit): the subtraction is exact, and the BF16
    # output is the sum's error, rounded by 2^-8 of itself
    w, x = _positive((rows, cols), 0.02, 1), _positive((tokens, cols), 1.0, 2)
    P = torch.cat([x.double() @ w[i:i + 1024].double().t() for i in range(0, rows, 1024)], dim=1)
    d = df11.compress_linear(w)
    y, = df11.decode_linear([d], [x], residuals=[-P.float()])
    parts = -(-cols // 512)
    bound = (1 + 2.0 ** -8) * (32 * 2.0 ** -23 + (parts + 1) * 2.0 ** -24)
    assert float((y.double().abs() / P).max()) <= bound
