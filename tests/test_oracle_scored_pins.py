"""Pins of the oracle's scored routing and dense 4-bit product (CPU only):
closed forms, a pure-Python enumeration of the choice, central differences
for the gradient, and the already pinned softmax routing."""

from __future__ import annotations

import itertools
import math

import numpy as np
import pytest

import moe_workloads as wl
from oracle import moe_oracle as mo


def logits_of(M, E, seed, spread=1.0):
    return (np.random.default_rng(seed).standard_normal((M, E)) * spread).astype(np.float32)


def test_softmax_rule_is_the_layers_own_routing():
    lay = wl.make_layer("toy", 3)
    r = mo.route(lay["x"], lay["w_router"], 2, True)
    ids = mo.select_ids(r["logits_f32"], 2, "softmax")
    assert np.array_equal(ids, r["topk_ids"])
    for renorm in (False, True):
        w = mo.select_weights(r["logits_f32"], ids, "softmax", renorm)
        assert np.abs(w - mo.weights_of(r["logits_f32"], ids, renorm)).max() < 1e-14


@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choice_by_enumeration(score, group_top):
    """The kept groups maximise the sum of group scores, the kept experts the
    sum of choice scores, over every combination."""
    M, E, G, kept, k = 12, 12, 4, 2, 3
    l = logits_of(M, E, 5)
    b = (np.random.default_rng(6).standard_normal(E) * 0.2).astype(np.float32)
    ids = mo.select_ids(l, k, score, b, G, kept, group_top)
    for t in range(M):
        if score == "sigmoid":
            s = [1.0 / (1.0 + math.exp(-float(v))) for v in l[t]]
        else:
            z = math.fsum(math.exp(float(v)) for v in l[t])
            s = [math.exp(float(v)) / z for v in l[t]]
        c = [s[e] + float(b[e]) for e in range(E)]
        size = E // G
        score_of = [math.fsum(sorted(c[g * size:(g + 1) * size])[-group_top:]) for g in range(G)]
        groups = max(itertools.combinations(range(G), kept),
                     key=lambda gs: math.fsum(score_of[g] for g in gs))
        members = [e for e in range(E) if e // size in groups]
        best = max(itertools.combinations(members, k), key=lambda es: math.fsum(c[e] for e in es))
        assert sorted(ids[t].tolist()) == sorted(best)
        assert all(c[a] >= c[b2] for a, b2 in zip(ids[t], ids[t][1:]))


def test_ties_masks_and_underflow():
    l = np.zeros((1, 6), dtype=np.float32)
    assert mo.select_ids(l, 3, "sigmoid").tolist() == [[0, 1, 2]]
    assert mo.select_ids(l, 2, "sigmoid", np.zeros(6, np.float32), 3, 1, 2).tolist() == [[0, 1]]
    l = np.full((1, 4), -np.inf, dtype=np.float32)
    ids = mo.select_ids(l, 2, "softmax")
    assert ids.tolist() == [[0, 1]]
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            assert mo.select_weights(l, ids, score, renorm).tolist() == [[0.0, 0.0]]
    # sigmoid(-900) underflows even in 64 bits; the ratio e^-1 does not
    l = np.array([[-900.0, -901.0]], dtype=np.float32)
    w = mo.select_weights(l, np.array([[0, 1]]), "sigmoid", True)
    assert np.allclose(w, [[1 / (1 + math.exp(-1)), math.exp(-1) / (1 + math.exp(-1))]], rtol=1e-12)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(score, renorm):
    M, E, k, scale = 3, 7, 3, 1.5
    l = logits_of(M, E, 9)
    ids = mo.select_ids(l, k, score)
    gw = logits_of(M, k, 10)
    got = mo.select_backward(l, ids, gw, score, renorm, scale)

    def loss(v):
        p = np.exp(mo.log_scores(v, score))
        s = np.take_along_axis(p, ids.astype(np.int64), axis=1)
        w = s / s.sum(axis=1, keepdims=True) if renorm else s
        return float((scale * w * gw).sum())

    h = 1e-5
    for t in range(M):
        for e in range(E):
            up, down = l.astype(np.float64), l.astype(np.float64)
            up[t, e] += h
            down[t, e] -= h
            # central differences: error h^2 * |third derivative| / 6 and 2^-52 / h
            assert abs((loss(up) - loss(down)) / (2 * h) - got[t, e]) < 1e-8


def test_linear_closed_forms():
    rng = np.random.default_rng(3)
    M, N, K, group = 3, 6, 64, 32
    x = wl.f32_to_bf16_bits(rng.standard_normal((M, K)).astype(np.float32))
    words = rng.integers(0, 2 ** 32, size=(N, K // 8), dtype=np.uint64).astype(np.uint32)
    one = wl.f32_to_bf16_bits(np.ones((N, K // group), dtype=np.float32))
    zero = np.zeros_like(one)
    X = mo.widen_bf16(x)
    # zero scales: every row is the sum of x; unit scales and no biases: the codes
    assert np.allclose(mo.linear_quantized(x, words, zero, one, group), X.sum(1, keepdims=True))
    codes = np.array([[(int(words[n, i // 8]) >> (4 * (i % 8))) & 15 for i in range(K)]
                      for n in range(N)], dtype=np.float64)
    y = mo.linear_quantized(x, words, one, zero, group)
    assert np.allclose(y, X @ codes.T)
    g = mo.linear_quantized(x, words, one, zero, group, gated=True)
    assert np.allclose(g, y[:, :3] / (1 + np.exp(-y[:, :3])) * y[:, 3:])
    rs = rng.random(M).astype(np.float32)
    out = mo.linear_quantized(x, words, one, zero, group, row_scale=rs, addend=x[:, :N])
    assert np.allclose(out, y * rs[:, None].astype(np.float64) + X[:, :N])


def test_planted_mistakes_are_caught():
    """Forms that differ from the definition differ in their results."""
    l = logits_of(64, 12, 1, 2.0)
    b = np.linspace(-0.3, 0.3, 12).astype(np.float32)
    ids = mo.select_ids(l, 3, "sigmoid", b, 4, 2, 2)
    assert not np.array_equal(ids, mo.select_ids(l, 3, "sigmoid", None, 4, 2, 2))
    assert not np.array_equal(ids, mo.select_ids(l, 3, "softmax", b, 4, 2, 2))
    assert not np.array_equal(ids, mo.select_ids(l, 3, "sigmoid", b, 4, 2, 1))
    assert not np.array_equal(ids, mo.select_ids(l, 3, "sigmoid", b))
    w = mo.select_weights(l, ids, "sigmoid", True)
    # the bias must not enter the weights
    s = 1 / (1 + np.exp(-l.astype(np.float64))) + b
    sb = np.take_along_axis(s, ids.astype(np.int64), axis=1)
    assert np.abs(w - sb / sb.sum(1, keepdims=True)).max() > 1e-2
