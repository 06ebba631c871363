"""Dense 4-bit products at the borders of their contract: rows of x that are
not finite."""

from __future__ import annotations

import numpy as np
import pytest

import moe_workloads as wl
from tests import helpers as h
from tests import test_gpu_qlinear as tl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("M", [1, 2, 3, 16, 40, 1030])
def test_rows_that_are_not_finite(M, bad, gated):
    """A result that is not finite in every output of such a row, whatever the
    signs of scale and bias, and every other row as without it."""
    import torch
    moe = tl._moe()
    N, K, group = (4096 if M == 1030 else 64), 512, 64       # the last: LDS tiles
    q, s, b = tl.matrix(N, K, group, 5)
    b[1::4] = wl.f32_to_bf16_bits(np.float32([0.5]))[0]       # b - 128 s > 0, as s
    s[2::4] |= 0x8000                                         # s < 0, b - 128 s > 0
    s[3::4] = 0
    b[3::8] = 0
    w = tl.to_device(q, s, b, group)
    x = h.dev_bf16(tl.rows(M, K, 6))
    good = moe.moe_linear_quantized(x, w, gated=gated)
    y = x.clone()
    y[M - 1, 7] = bad
    got = moe.moe_linear_quantized(y, w, gated=gated)
    torch.cuda.synchronize()
    assert torch.isfinite(good).all()
    assert not torch.isfinite(got[M - 1]).any()
    assert torch.equal(got[:M - 1], good[:M - 1])
