"""The log probabilities' gradient of rows that a large negative number, not
-inf, rules out from end to end."""

from __future__ import annotations

import numpy as np
import pytest

from tests import test_gpu_logprobs as tl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", tl.DTYPES)
@pytest.mark.parametrize("low", [-3e7, -1e9, -1e20, -1e30, "lowest"])
@pytest.mark.parametrize("V", [2, 300, 70001])
def test_gradient_of_a_row_ruled_out_is_zero(V, low, dtype):
    """fp32's step is 2 or more from 2^24 on: such a row's lse says nothing of
    how many logits share it, e^(l - lse) is 1 for each of them."""
    v = tl.LOWEST[dtype] if low == "lowest" else low
    l = tl.draw(4, V, 21)
    l[1, :] = v
    l[2, 1:] = v
    for entropy in (True, False):
        got, _, _, _ = tl.check_grad(l, dtype, np.array([V - 1, 0, 0, 1]), entropy)
        assert not got[1].any()
        assert got[0].any() and got[3].any()


@pytest.mark.parametrize("dtype", tl.DTYPES)
@pytest.mark.parametrize("low", [-1e4, -3e5, -1.6e7])
def test_gradient_of_logits_far_below_0_sums_to_0(low, dtype):
    """Above -2^24 the gradient is formed from lse as it is: softmax's sum is 1
    but for lse's rounding, off by 2^-24 |lse| at most, so that the gradient's
    sum is g (1 - e^d) with |d| of that size."""
    V, U = 1000, tl.U
    l = np.full((2, V), low, np.float32)
    got, l, g, _ = tl.check_grad(l, dtype, np.array([3, 999]), entropy=False)
    d = U * abs(float(l[0, 0])) + 1e-5       # and the forward pass's own few roundings
    p = np.exp(d)
    # each of V gradients rounded to the type once more
    half = 2.0 ** -8 if dtype == "bfloat16" else U
    assert np.all(np.abs(got.sum(axis=1)) <= np.abs(g) * (p - 1 + 2 * p * (half + 50 * U)))
    assert got.all()
