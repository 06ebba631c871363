"""Scored routing, its gradient and the dense 4-bit product at the batch sizes
that choose each of their kernels: lanes per token and experts per lane of the
routing kernels, row tiles and both widths of the LDS tiles of the products.
The inputs hold what the small tests hold (ties, masked rows, neighbours one
rounding apart, rows that are not finite), between ordinary rows.
"""

from __future__ import annotations

import numpy as np
import pytest

from oracle import moe_oracle as mo
from tests import helpers as h
from tests import test_gpu_qlinear as tl
from tests import test_gpu_select as ts

pytestmark = pytest.mark.gpu

INF = np.float32(np.inf)


def batch(M, E, k, seed):
    """Ordinary rows, and in every 64 of them one each of: few values, one
    value, half masked, all but k masked, all masked, the type's lowest value,
    two logits one fp32 step apart at the border of the choice."""
    rng = np.random.default_rng(seed)
    l = ts.draw(M, E, seed)
    l[1::64] = rng.integers(-1, 2, size=l[1::64].shape)
    l[5::64] = 0.25
    l[9::64, ::2] = -INF
    l[20::64, k:] = -INF
    l[21::64] = -INF
    l[33::64] = np.finfo(np.float32).min
    if k < E:
        near = l[40::64]
        order = np.argsort(-near, axis=1)
        at = np.arange(near.shape[0])
        near[at, order[:, k]] = np.nextafter(near[at, order[:, k - 1]], np.float32(-9))
        l[40::64] = near
    return l


@pytest.mark.parametrize("M,E,k,score,renorm,bias,G,kept,top", [
    # sixteen lanes a token: 4, 8, 16, 32 experts a lane, whole fours and not
    (300, 64, 12, "sigmoid", True, True, 1, 1, 1),
    (70001, 62, 4, "softmax", False, True, 1, 1, 1),
    (8300, 128, 12, "softmax", True, False, 1, 1, 1),
    (8300, 126, 8, "sigmoid", False, True, 1, 1, 1),
    (16500, 256, 8, "sigmoid", True, True, 8, 4, 2),
    (16500, 256, 3, "softmax", True, True, 8, 1, 1),
    (16500, 250, 12, "softmax", True, True, 1, 1, 1),
    (33001, 512, 10, "sigmoid", True, True, 1, 1, 1),
    (33001, 510, 8, "softmax", False, False, 5, 2, 2),
    # 32 lanes: 4, 8, 16 experts a lane
    (1500, 100, 13, "softmax", True, True, 1, 1, 1),
    (700, 126, 20, "sigmoid", True, False, 1, 1, 1),
    (16400, 256, 26, "sigmoid", True, True, 8, 4, 2),
    (700, 250, 17, "softmax", False, True, 5, 4, 1),
    (9000, 512, 8, "softmax", True, True, 4, 1, 1),
    (1500, 510, 26, "sigmoid", False, True, 1, 1, 1),
    # a wave: 4, 8, 16 experts a lane; fewer open lanes than top_k
    (3000, 124, 32, "softmax", True, True, 1, 1, 1),
    (700, 512, 29, "sigmoid", True, True, 8, 3, 1),
    (300, 480, 30, "softmax", True, False, 24, 8, 1),
    (300, 510, 32, "softmax", False, True, 2, 1, 2),
])
def test_select_variants(M, E, k, score, renorm, bias, G, kept, top):
    """A sample of the rows against the oracle; every row against the same row
    in a batch of 600, where another variant chooses."""
    moe = ts._moe()
    l, b = batch(M, E, k, E + k), ts.steps(E, E) if bias else None
    r = moe.Routing(k, score=score, renormalize=renorm, select_bias=None if b is None else h.dev_f32(b),
                    n_group=G, topk_group=kept, group_top=top, scale=2.5)
    ids, w = ts.run_select(l, r)
    at = np.unique(np.concatenate([np.arange(min(M, 260)), np.arange(M - 70, M),
                                   np.random.default_rng(9).integers(0, M, 200)]))
    ref = mo.select_ids(l[at], k, score, b, G, kept, top)
    assert np.array_equal(ids[at], ref)
    wr = mo.select_weights(l[at], ref, score, renorm, 2.5)
    tol = ts.rel_tol(l, k)
    assert np.all(np.abs(w[at] - wr) <= tol * np.abs(wr) + 2.0 ** -126 * 2.5)
    for m in range(0, M, 600):
        part, pw = ts.run_select(l[m:m + 600], r)
        assert np.array_equal(ids[m:m + 600], part)
        assert np.all(np.abs(w[m:m + 600] - pw) <= 2 * tol * np.abs(pw) + 2.0 ** -125 * 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_masked_experts_that_a_bias_chooses(score, renorm):
    """Distinct biases choose among experts whose logits are -inf: rows where
    every one is, and where the bias passes over the finite ones."""
    E, k = 64, 4
    l = ts.draw(6, E, 4)
    l[1] = -INF
    l[2, :E - 8] = -INF
    l[3, 8:] = -INF
    bias = np.arange(E, 0, -1, dtype=np.float32)
    ids, w = ts.check(l, k, score, renorm, bias)
    assert np.all(ids == np.arange(k)) and np.all(w[1:3] == 0.0)
    ts.check(l, k, score, renorm, bias, 8, 4, 2)


def test_more_undecided_rows_than_a_wave_lists_at_once():
    """Ties in a biased softmax are done over one by one, 64 of a wave's rows
    at a time: here a wave has about 80."""
    l = np.random.default_rng(3).integers(-1, 2, size=(800_001, 8)).astype(np.float32)
    moe = ts._moe()
    ids, w = ts.run_select(l, moe.Routing(2, select_bias=h.dev_f32(np.zeros(8, np.float32))))
    ref = np.argsort(-l, axis=1, kind="stable")[:, :2]
    assert np.array_equal(ids, ref)
    e = np.exp(np.take_along_axis(l.astype(np.float64), ref, axis=1))
    assert np.all(np.abs(w - e / e.sum(1, keepdims=True)) <= ts.rel_tol(l, 2))


@pytest.mark.parametrize("M,E,k,score,renorm", [
    (300, 64, 16, "softmax", False), (20001, 62, 4, "softmax", False), (8300, 128, 8, "sigmoid", True),
    (33001, 512, 10, "sigmoid", True), (33001, 510, 16, "softmax", True),
    (9000, 512, 32, "softmax", False), (2000, 510, 10, "sigmoid", False)])
def test_backward_variants(M, E, k, score, renorm):
    l = batch(M, E, k, E)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    ids[2::64, 1] = ids[2::64, 0]
    ids[3::64, 0] = -1
    ids[4::64, k - 1] = E
    keep = np.ones(M, bool)
    keep[3::64] = keep[4::64] = False
    g = ts.draw(M, k, 5)
    moe = ts._moe()
    got = ts.run_backward(l, ids, g, moe.Routing(k, score=score, renormalize=renorm, scale=2.5))
    ref = mo.select_backward(l[keep], ids[keep], g[keep], score, renorm, 2.5)
    # as for the small batches: factors <= 1 with scale * g, errors of the
    # weights and of sums of k terms
    tol = (3 * ts.rel_tol(l, k) + 2 * k * 2.0 ** -23) * 2.5 * np.abs(g).sum(1, keepdims=True)
    assert np.all(np.abs(got[keep] - ref) <= tol[keep] + 2.0 ** -126)
    # a slot that names no expert takes no part
    for t, used in [(t, np.arange(1, k)) for t in range(3, M, 64)][:20] + \
                   [(t, np.arange(k - 1)) for t in range(4, M, 64)][:20]:
        one = mo.select_backward(l[t:t + 1], ids[t:t + 1, used], g[t:t + 1, used], score, renorm, 2.5)
        assert np.all(np.abs(got[t] - one[0]) <= tol[t] + 2.0 ** -126)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,gated,scaled,added,in_place", [
    (300, 5632, False, False, False, False), (300, 5634, True, True, True, True),
    (321, 5633, False, True, True, True),
    (1030, 4100, False, False, True, False), (1030, 4098, True, True, False, False)])
def test_product_tiles(M, N, gated, scaled, added, in_place, group):
    for K in (group, 256, 384, 896):
        tl.check(M, N, K, group, K, gated, scaled, added, in_place)


@pytest.mark.parametrize("M,N,K", [(8, 40000, 256), (3, 9000, 1024), (16, 33000, 1024), (40, 5000, 512)])
def test_product_rows(M, N, K):
    for group, gated in ((32, True), (64, False), (128, True)):
        tl.check(M, N, K, group, M, gated, scaled=True)


@pytest.mark.parametrize("M,N", [(300, 5632), (1030, 4100)])
def test_product_tiles_keep_rows_apart_and_replay(M, N):
    """A row that is not finite stays alone; captured calls between eager
    ones, and two streams at once, give the eager result bit for bit."""
    import torch
    moe = tl._moe()
    K, group = 896, 128
    ws = [tl.to_device(*tl.matrix(N, K, group, 20 + i), group) for i in range(2)]
    x = h.dev_bf16(tl.rows(M, K, 22))
    want = [moe.moe_linear_quantized(x, w) for w in ws]
    y = x.clone()
    y[M - 2, 7] = float("inf")
    y[70, K - 1] = float("nan")
    bad = moe.moe_linear_quantized(y, ws[0])
    torch.cuda.synchronize()
    assert torch.isnan(bad[70]).all() and torch.isnan(bad[M - 2]).all()
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[70] = keep[M - 2] = False
    assert torch.equal(bad[keep], want[0][keep])
    graphs = []
    for w in ws:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = moe.moe_linear_quantized(x, w)
        graphs.append((g, out))
    for _ in range(3):
        for (g, out), exp in zip(graphs, want):
            out.zero_()
            g.replay()
            again = moe.moe_linear_quantized(x, ws[0])
            torch.cuda.synchronize()
            assert torch.equal(out, exp) and torch.equal(again, want[0])
    streams = [torch.cuda.Stream() for _ in ws]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    out = [[moe.moe_linear_quantized(x, w, stream=s) for w, s in zip(ws, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for rnd in out for a, b in zip(rnd, want))


def test_outputs_for_another_stream_do_not_take_the_current_ones_memory():
    """What the current stream freed it may still be using: a tensor made for
    a call on another stream comes from elsewhere."""
    import torch
    moe = ts._moe()
    E, k, M = 64, 4, 1 << 18
    l = h.dev_f32(ts.draw(M, E, 1))
    r = moe.Routing(k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    before = [torch.empty((M, k), dtype=torch.int32, device="cuda"),
              torch.empty((M, k), dtype=torch.float32, device="cuda")]
    used = {t.data_ptr() for t in before}
    del before
    ids, w = moe.moe_select(l, r, stream=s)
    assert not {ids.data_ptr(), w.data_ptr()} & used
    torch.cuda.current_stream().wait_stream(s)
    a, b = moe.moe_select(l, r)
    assert torch.equal(ids, a) and torch.equal(w, b)
