"""Dense 4-bit products at the borders of their contract: rows of x that are
not finite, few weight rows for many tokens, more slices of K than waves."""

from __future__ import annotations

import numpy as np
import pytest

import moe_workloads as wl
from oracle import moe_oracle as mo
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


def sampled(M, N, K, group, gated=False, seed=7):
    """A product checked on a sample of its tokens, the rows behind it
    untouched."""
    import torch
    moe = tl._moe()
    q, s, b = tl.matrix(N, K, group, seed)
    x = tl.rows(M, K, seed + 1)
    n_out = N // 2 if gated else N
    buf = torch.full((M * n_out + 16,), -7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:M * n_out].view(M, n_out)
    moe.moe_linear_quantized(h.dev_bf16(x), tl.to_device(q, s, b, group), gated=gated, out=out)
    torch.cuda.synchronize()
    assert (buf[M * n_out:] == -7.0).all()
    r = np.unique(np.concatenate([[0, M - 1], np.random.default_rng(seed).integers(0, M, 60)]))
    ref = mo.linear_quantized(x[r], q, s, b, group, gated)
    e = tl.error_bound(x[r], q, s, b, group, gated, None, None)
    got = h.host_bf16_to_f64(out[torch.from_numpy(r).cuda()])
    assert np.all(np.abs(got - ref) <= e + (np.abs(ref) + e) * 2.0 ** -8)


@pytest.mark.parametrize("M,N,K,group,gated", [
    (16384, 16, 512, 64, False), (16385, 64, 512, 32, False), (32768, 64, 512, 128, False),
    (16384, 32, 256, 64, True), (20000, 2, 512, 64, True), (65536, 16, 64, 64, False),
    (16400, 1, 2048, 128, False)])
def test_few_weight_rows_for_many_tokens(M, N, K, group, gated):
    """Fewer tiles of weight rows than a workgroup would walk."""
    sampled(M, N, K, group, gated)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("K,group", [(16384 + 32, 32), (18432, 128), (32768 + 64, 64), (40960, 128)])
@pytest.mark.parametrize("M", [1, 2, 16, 33])
def test_more_slices_of_k_than_waves(M, K, group, gated):
    tl.check(M, 24, K, group, K, gated, True, True)
