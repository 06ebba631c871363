"""Borders of the dense operators: rows that are not finite and what they may
reach, the largest vocabulary, grids of more than one layer, operands past 2^31
elements."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import dense_oracle as do
from oracle import moe_oracle as mo
from tests import helpers as h
from tests import test_gpu_adapters as ta
from tests import test_gpu_gated as tg
from tests import test_gpu_logprobs as tl

pytestmark = pytest.mark.gpu

BAD = [float("nan"), float("inf"), float("-inf")]


@pytest.mark.parametrize("M", [1, 4, 5, 20, 40, 70, 300])
@pytest.mark.parametrize("H", [200, 2048])
def test_gated_row_that_is_not_finite(H, M):
    """Each of its own results is not finite (no weight is 0: gate and up are
    both infinite or NaN), and every other row keeps its bits."""
    import torch
    moe = tg._moe()
    x, w, _ = tg.inputs(M, H, 72, 5)
    x, w = h.dev_bf16(x), h.dev_bf16(w)
    w[w == 0] = 0.5
    good = moe.moe_linear_gated(x, w)
    for bad in BAD:
        for m in {0, M // 2, M - 1}:
            y = x.clone()
            y[m, H - 1] = bad
            out = moe.moe_linear_gated(y, w)
            torch.cuda.synchronize()
            assert not torch.isfinite(out[m]).any()
            rest = torch.arange(M, device="cuda") != m
            assert torch.equal(out[rest], good[rest])


@pytest.mark.parametrize("M", [2, 5, 16, 17, 64, 65, 300])
@pytest.mark.parametrize("where", ["x", "grad_out"])
def test_gated_gradient_row_that_is_not_finite(where, M):
    """grad_x's row is its own; grad_w13 sums over the rows."""
    import torch
    moe = tg._moe()
    H, I = 200, 72
    x, w, d = (h.dev_bf16(t) for t in tg.inputs(M, H, I, 6))
    w[w == 0] = 0.5
    good, _ = moe.moe_linear_gated_backward(x, w, d)
    for bad in BAD:
        for m in {0, M // 2, M - 1}:
            y, e = x.clone(), d.clone()
            if where == "x":
                y[m, H - 1] = bad
            else:
                e[m, I - 1] = bad
            gx, gw = moe.moe_linear_gated_backward(y, w, e)
            torch.cuda.synchronize()
            assert not torch.isfinite(gx[m]).any()
            rest = torch.arange(M, device="cuda") != m
            assert torch.equal(gx[rest], good[rest])
            # every feature's sums hold the bad row's term (x: each of them, d: one)
            hit = gw if where == "x" else gw[[I - 1, 2 * I - 1]]
            assert not torch.isfinite(hit).any()


@pytest.mark.parametrize("dtype", tl.DTYPES)
def test_logprobs_token_outside_a_row_that_is_not_finite(dtype):
    """A token outside the vocabulary has log probability 0 in any row."""
    l = tl.draw(4, 500, 3)
    l[0, 7], l[1, 8], l[2, :] = np.nan, np.inf, -np.inf
    got = tl.check(l, dtype, 4, np.array([-1, 500, 2 ** 31 - 1, -2 ** 31]))
    assert not got[0].any()


@pytest.mark.parametrize("dtype", tl.DTYPES)
def test_logprobs_largest_vocabulary(dtype):
    """Ties on both sides of the highest bit of an id, and at the last ones."""
    V = 2 ** 19
    rng = np.random.default_rng(1)
    l = np.full((5, V), -3.5, np.float32)
    l[0, 262144 - 16:] = 2.0                       # the lower ids of many
    l[1, rng.integers(262144, V, 12)] = 2.0
    l[1, rng.integers(0, 262144, 9)] = 2.0
    l[2, V - 20:] = 2.0
    l[3] = tl.draw(1, V, 4)
    l[4, 262144 - 5:262144 + 5] = 1.0
    tokens = np.array([262144, 262143, V - 1, V - 2, 0])
    for top in (1, 20, 32):
        tl.check(l, dtype, top, tokens)
    tl.check_grad(l, dtype, tokens)


def test_adapters_more_units_than_a_grid_layer():
    """8 windows of 128 + 4097 units: a second layer of the grid."""
    ta.check(65536, 4096, 8, 8, 8, seed=3)
    ta.check(65536, 4096, 8, 8, 16, seed=4, gated=True)


def test_gated_past_32_bits():
    """out, grad_out and the workspace have more than 2^31 elements, and rows
    on both sides of them.  Of the other rows the gradient that comes in is 0."""
    import torch
    moe = tg._moe()
    M, H, I = 1050003, 16, 2056
    pick = np.array([0, 1, 261184, 522247, 1044493, 1044494, 1048575, 1048576, M - 2, M - 1])
    x, w, d = tg.inputs(len(pick), H, I, 8)
    at = torch.from_numpy(pick).cuda()
    dx = torch.ones((M, H), dtype=torch.bfloat16, device="cuda")
    dx[at] = h.dev_bf16(x)
    dw = h.dev_bf16(w)
    out = moe.moe_linear_gated(dx, dw)
    X, W, g, u, eg, eu = tg.parts(x, w)
    err = np.abs(h.host_bf16_to_f64(out[at]) - do.gated(X, W))
    assert np.all(err <= tg.act_bound(g, u, eg, eu))
    dd = out.zero_()
    dd[at] = h.dev_bf16(d)
    gx, gw = moe.moe_linear_gated_backward(dx, dw, dd)
    want = do.gated_backward(X, W, mo.widen_bf16(d).astype(np.float64))
    (_, bx), _ = tg.grad_bounds(x, w, d)
    assert np.all(np.abs(h.host_bf16_to_f64(gx[at]) - want[0]) <= bx)
    gx[at] = 0
    assert not gx.any()
    # the other rows add exact zeros, which round nothing
    _, (_, bw) = tg.grad_bounds(x, w, d)
    assert np.all(np.abs(h.host_bf16_to_f64(gw) - want[1]) <= bw)


def test_adapters_past_32_bits():
    import torch
    moe = ta._moe()
    M, S, R, K, N = 524300, 3, 8, 16, 4104
    pick = np.array([0, 1, 261624, 523264, 523265, 523266, M - 2, M - 1])
    d = ta.inputs(len(pick), S, R, K, N, 5)
    d["random"][:] = [0, 1, 2, 0, -1, 1, 2, 0]
    at = torch.from_numpy(pick).cuda()
    x = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    x[at] = h.dev_bf16(d["x"])
    slots = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    slots[at] = h.dev_i32(d["random"])
    y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    y[at] = h.dev_bf16(d["addend"])
    ad = dict(a=h.dev_bf16(d["a"]), b=h.dev_bf16(d["b"]), scales=h.dev_f32(d["scales"]))
    out = moe.moe_linear_adapters(x, ad, slots, addend=y)
    assert moe.moe_linear_adapters(x, ad, slots, addend=y, out=y) is y
    ref, bound = ta.reference(d, d["random"], True, True, False)
    for t in (out, y):
        assert np.all(np.abs(h.host_bf16_to_f64(t[at]) - ref) <= bound)
        t[at] = 0
        assert not t.any()
