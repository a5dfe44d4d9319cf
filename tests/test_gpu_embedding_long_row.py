"""Rows that end next to element 2^32: the lookup's segments of them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

df11 = pytest.importorskip("huffman_decode_df11_b200")


@pytest.mark.parametrize("dim", [2 ** 32 - 96, 2 ** 32 - 5])
def test_a_single_row_of_nearly_two_to_the_32_elements(dim):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    # a pattern of period 1009 (prime), so that a part at another place shows
    part = torch.randn(1009, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    w = part.repeat(-(-dim // 1009))[:dim].view(1, dim)
    d = df11.compress_on_device(w)
    out = torch.full((2, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    err = df11.new_error_word()
    df11.decode_embedding(d, torch.tensor([0, 1], device="cuda"), out, err=err)  # 1: outside the table
    torch.cuda.synchronize()
    with pytest.raises(df11.Df11Error, match="INDEX"):
        df11.check_device_error(err)
    assert torch.equal(out[0].view(torch.int16), w[0].view(torch.int16))
    assert not out[1].any()
    del w, d, out
    torch.cuda.empty_cache()
