"""Scored routing where a plain fp32 evaluation goes wrong: masks of the
type's lowest value, group sums of large biases that cancel, NaN among the
chosen experts, a single renormalized weight, saturated scores."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import moe_oracle as mo
from tests import helpers as h
from tests import test_gpu_select as ts

pytestmark = pytest.mark.gpu

INF = np.float32(np.inf)
LOWEST = np.finfo(np.float32).min


@pytest.mark.parametrize("low", [-INF, LOWEST, np.float32(-1e9)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_group_sums_with_masking_biases(score, low):
    """Biases that mask experts: one expert left in some groups, none in
    others, a group's sum past the type's lowest value."""
    E, G = 96, 8
    l = ts.draw(300, E, 17)
    bias = ts.steps(E, 18)
    bias[1:12] = low                        # one expert of group 0 stays
    bias[12:24] = low                       # none of group 1
    bias[24:35] = low
    bias[40:44] = low
    for kept in (1, 3, 6, 7, 8):
        for top in (1, 2):
            ts.check(l, 8 if kept > 1 else 2, score, True, bias, G, kept, top)


@pytest.mark.parametrize("low", [-INF, LOWEST, np.float32(-1e9)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,M", [(33, 1, 9), (60, 1, 4000), (510, 1, 700), (510, 5, 9), (3, 1, 5)])
def test_masking_biases_where_lanes_have_spare_experts(E, G, M, score, low):
    """The choice reaches masked experts, and lanes hold places for experts
    that do not exist: those are never chosen."""
    bias = ts.steps(E, 19)
    bias[2:E // G] = low
    if G > 1:
        bias[E // G:] = low
    l = ts.draw(M, E, 20)
    k = min(E, 6)
    ids, _ = ts.check(l, k, score, True, bias, G, min(G, 2), 1)
    assert np.all((ids >= 0) & (ids < E))


# ---------------------------------------------------------------------------
# group sums of large biases that cancel
# ---------------------------------------------------------------------------

def cancelling(score, B, G, M, seed):
    """M rows of G groups of two whose biases are +B and -B: a group's sum is
    s0 + s1, all of them within 2e-5 of each other, and each group's c was
    rounded at the magnitude B.  Rows whose two sums at the border of the kept
    groups lie closer than 2e-7 are left out: below B = 1e4 double precision
    tells the others apart (its c rounds by 2^-53 B = 1.1e-12)."""
    rng = np.random.default_rng(seed)
    n = 3 * M
    if score == "sigmoid":
        total = 1.0
    else:
        total = 1.0 / G
    s0 = total * rng.uniform(0.2, 0.8, size=(n, G))
    s1 = total + rng.uniform(-1e-5, 1e-5, size=(n, G)) - s0
    s = np.stack([s0, s1], axis=2).reshape(n, 2 * G)
    l = np.log(s / (1.0 - s)) if score == "sigmoid" else np.log(s)
    l = l.astype(np.float32)
    sums = np.sort(np.exp(mo.log_scores(l, score)).reshape(n, G, 2).sum(2), axis=1)
    kept = max(1, G // 3)
    l = l[sums[:, G - kept] - sums[:, G - kept - 1] > 2e-7][:M]
    assert l.shape[0] == M
    return l, np.tile(np.float32([B, -B]), G), kept


@pytest.mark.parametrize("M", [700, 4096])
@pytest.mark.parametrize("G", [2, 8, 16])
@pytest.mark.parametrize("B", [16.0, 100.0, 1e4])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_group_sums_of_cancelling_biases(score, B, G, M):
    l, bias, kept = cancelling(score, B, G, M, int(B) + G)
    ts.check(l, kept, score, True, bias, G, kept, 2)


# ---------------------------------------------------------------------------
# NaN among the chosen
# ---------------------------------------------------------------------------

def by_formula(l, ids, score, renorm):
    """Weights as the formula has them in float64.  Renormalized softmax
    weights are formed from the chosen logits alone."""
    l = l.astype(np.float64)
    lk = np.take_along_axis(l, ids.astype(np.int64), axis=1)
    with np.errstate(invalid="ignore"):
        if renorm and score == "softmax":
            m = np.where(np.isnan(lk), -np.inf, lk).max(axis=1, keepdims=True)
            s = np.exp(lk - np.where(np.isneginf(m), 0.0, m))
        elif score == "softmax":
            s = np.exp(lk) / np.exp(l).sum(axis=1, keepdims=True)
        else:
            s = 1.0 / (1.0 + np.exp(-lk))
        w = s / s.sum(axis=1, keepdims=True) if renorm else s
    # a chosen row of -inf alone: 0
    return np.where(np.isneginf(lk).all(axis=1, keepdims=True), 0.0, w)


@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_chosen_nan_reaches_the_weights(score, renorm, biased, G):
    """Rows with too few numbers to choose from: NaN logits are chosen last,
    and their weights, and the gradient through them, are NaN, never 0."""
    moe = ts._moe()
    E, k, nan = 64, 5, np.float32(np.nan)
    l = ts.draw(8, E, 31)
    l[1] = nan
    l[2, 3:] = nan
    l[3] = nan
    l[3, 7] = l[3, 40] = -INF
    l[4] = nan
    l[4, 9], l[4, 41] = 0.5, -INF
    l[6] = -INF
    r = moe.Routing(k, score=score, renormalize=renorm, n_group=G, topk_group=min(G, 2), scale=2.5,
                    select_bias=h.dev_f32(ts.steps(E, 32)) if biased else None)
    ids, w = ts.run_select(l, r)
    assert all(len(set(row)) == k for row in ids.tolist())
    assert np.all((ids >= 0) & (ids < E))
    want = 2.5 * by_formula(l, ids, score, renorm)
    lk = np.take_along_axis(l, ids.astype(np.int64), axis=1)
    assert np.isnan(lk[[1, 2, 3, 4]]).any(axis=1).all()
    assert np.array_equal(np.isnan(w), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.all(np.abs(w - want)[ok] <= ts.rel_tol(l, k) * np.abs(want[ok]) + 2.0 ** -126 * 2.5)
    g = ts.draw(8, k, 33)
    got = ts.run_backward(l, ids, g, r)
    at = np.take_along_axis(got, ids.astype(np.int64), axis=1)
    if renorm or score == "softmax":
        # every chosen expert's weight holds the NaN
        assert np.isnan(at[[1, 2, 3, 4]]).all()
    else:
        assert np.array_equal(np.isnan(at), np.isnan(lk))
    if renorm or score == "sigmoid":
        rest = got.copy()
        np.put_along_axis(rest, ids.astype(np.int64), 0.0, axis=1)
        assert np.all(rest == 0.0)
    fine = [0, 5, 7]
    ref = mo.select_backward(l[fine], ids[fine], g[fine], score, renorm, 2.5)
    tol = (3 * ts.rel_tol(l, k) + 2 * k * 2.0 ** -23) * 2.5 * np.abs(g[fine]).sum(1, keepdims=True)
    assert np.all(np.abs(got[fine] - ref) <= tol + 2.0 ** -126)
    assert np.all(got[6] == 0.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [1, 60, 512])
def test_gradient_of_one_renormalized_weight_is_zero(E, score):
    """w = scale * s / s is constant: its gradient is 0, not a rounding."""
    moe = ts._moe()
    l = ts.draw(600, E, 41, 3.0)
    ids = mo.select_ids(l, 1, score)
    got = ts.run_backward(l, ids, ts.draw(600, 1, 42), moe.Routing(1, score=score, scale=2.5))
    assert np.all(got == 0.0)


@pytest.mark.parametrize("G,kept", [(1, 1), (8, 3)])
@pytest.mark.parametrize("shift", [300.0, -1000.0])
def test_saturated_scores_are_ordered_by_their_logits(shift, G, kept):
    """Sigmoid scores that all round to 1, or to 0: without a bias experts and
    groups go by the logits, as a softmax's scores of the same logits do."""
    moe = ts._moe()
    l = ts.draw(70, 128, 51, 3.0) + np.float32(shift)
    ids, w = ts.run_select(l, moe.Routing(6, score="sigmoid", n_group=G, topk_group=kept))
    assert np.array_equal(ids, mo.select_ids(l, 6, "softmax", None, G, kept, 1))
    wr = mo.select_weights(l, ids, "sigmoid", True)
    assert np.all(np.abs(w - wr) <= ts.rel_tol(l, 6) * wr)
