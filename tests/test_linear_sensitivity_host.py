"""What the product's tests on whole numbers can see, on the CPU: in data like theirs no group of
16 columns can be left out, counted twice or exchanged with the next one without a change."""
import numpy as np
import pytest


@pytest.mark.parametrize("cols", [12288, 49152, 80000])
def test_every_group_of_columns_counts(cols):
    rng = np.random.default_rng(1)
    w, x = rng.integers(-7, 8, (16, cols)), rng.integers(-7, 8, (1, cols))
    groups = (w * x).reshape(16, cols // 16, 16).sum(axis=2)
    # the weights of group g + 1 on the activations of group g
    v, u = w.reshape(16, -1, 16), x.reshape(1, -1, 16)
    exchanged = ((v[:, 1:] - v[:, :-1]) * (u[:, :-1] - u[:, 1:])).sum(axis=2)
    assert np.all(np.any(groups != 0, axis=0)) and np.all(np.any(exchanged != 0, axis=0))
    assert np.abs(w * x).sum(axis=1).max() < 2 ** 24  # a row's sums, in any order, are exact in fp32
