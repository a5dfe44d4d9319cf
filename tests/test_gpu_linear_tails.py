"""The activations far out in their tails, relative to their value.

silu(v) = v e e / (1 + e e) with e = exp(-|v|/2): exp within 2 units (4 half units of 2^-24), twice,
two products, a sum and a division within 2 units, 15 half units in all; 16 allowed.  The tanh form's
exponent t comes from some 7 roundings of half a unit, so its relative error counts |t| times:
16 + 8 |t| half units.  gelu(v) = v/2 erfc(x), x = -v/sqrt(2) with 2 half units of error, which
count 2 x^2 + 1 times, and erfc within 4 units: 16 + 8 x^2.  Below the smallest normal number a
product and a quotient may be off by half of its step each: 2^-148.  BF16 outputs are rounded
by 2^-8 of the value, or half of their smallest step, 2^-134.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

df11 = pytest.importorskip("huffman_decode_df11_b200")

VALUES = [-100.0, -90.0, -88.5, -87.5, -87.0, -60.0, -13.0, -12.0, -10.5, -10.375, -9.0, -3.0, -0.5,
          -1e-30, -0.0, 1e-30, 0.25, 2.0, 10.0, 80.0, 88.5, 300.0, 3e38]


def _exact(name, v):
    """The activation in 64 bits, and the half units that its evaluation may be off by."""
    if name == "silu":
        return v * torch.sigmoid(v), 16 + 0 * v
    if name == "gelu_tanh":
        t = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        return v * torch.sigmoid(t), torch.where(t < 0, 16 + 8 * t.abs(), 16.0)
    x = -v / math.sqrt(2)
    return 0.5 * v * torch.special.erfc(x), torch.where(x > 0, 16 + 8 * x * x, 16.0)


@pytest.mark.parametrize("activation", ["silu", "gelu_tanh", "gelu"])
@pytest.mark.parametrize("tokens", [len(VALUES), 2 * len(VALUES)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_tails(activation, tokens, out):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    w = torch.zeros(16, 64, dtype=torch.bfloat16)
    w[3, 5] = 1.0                                       # the products are x itself
    x = torch.zeros(tokens, 64, dtype=torch.bfloat16)
    x[:, 5] = torch.tensor(VALUES * 2)[:tokens].to(torch.bfloat16)
    y, = df11.decode_linear([df11.compress_linear(w.cuda())], [x.cuda()], activations=[activation],
                            out_dtype=out)
    y = y.cpu().double()[:, 3]
    want, units = _exact(activation, x[:, 5].double())
    bound = units * 2.0 ** -24 * want.abs() + 2.0 ** -148
    if out == torch.bfloat16:
        bound = bound + torch.clamp(2.0 ** -8 * want.abs(), min=2.0 ** -134)
    off = (y - want).abs()
    assert torch.all(off <= bound), [(float(v), float(a), float(b)) for v, a, b, o, e in
                                     zip(x[:, 5], y, want, off, bound) if not o <= e]
