"""Borders of the dense operators' float64 oracle."""

from __future__ import annotations

import numpy as np

from oracle import dense_oracle as do


def test_gradient_of_a_row_far_below_0():
    l = np.full((2, 4), -(2.0 ** 24) - 8.0, np.float32)
    l[1] += 16.0
    lse = l[:, 0].astype(np.float32)
    d = do.token_logprobs_backward(l, np.array([0, 0]), lse, np.zeros(2), np.ones(2), np.zeros(2))
    assert not d[0].any() and d[1].any()
