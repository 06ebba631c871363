"""Scored routing on the GPU (moe_select, moe_select_backward,
moe_route_scored) against the float64 oracle."""

from __future__ import annotations

import numpy as np
import pytest

import moe_workloads as wl
from oracle import moe_oracle as mo
from tests import helpers as h

pytestmark = pytest.mark.gpu

INF = float("inf")


def _moe():
    import mixture_experts_ffn_renorm_amd as moe
    return moe


def draw(M, E, seed, spread=1.0):
    return (np.random.default_rng(seed).standard_normal((M, E)) * spread).astype(np.float32)


def steps(E, seed, step=1e-3, n=30):
    """A balance bias: a sum of steps up and down."""
    return (np.round(np.random.default_rng(seed).standard_normal(E) * n) * step).astype(np.float32)


def rel_tol(l, k):
    """Relative error of one weight: an exponential of a difference of logits
    rounds its argument by 2^-24 of |l_i - l_j| <= 2 max|l| and itself by an
    ulp; sums of k (or, over all experts, 8 per lane and 6 steps) positive
    terms and a quotient add at most k + 20 half ulps.  Logits beyond 2000
    count only as masks: they score 0 beside the others, or, a whole row of
    one value, differ by 0."""
    fin = np.abs(l[np.abs(l) <= 2000])
    return (2.0 * (fin.max() if fin.size else 0.0) + k + 20) * 2.0 ** -23


def run_select(l, routing, tail=3):
    """ids and weights of a batch; the rows behind it must stay untouched."""
    import torch
    moe = _moe()
    M, k = l.shape[0], routing.top_k
    ids = torch.full((M + tail, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((M + tail, k), -7.0, dtype=torch.float32, device="cuda")
    moe.moe_select(h.dev_f32(l), routing, topk_ids=ids[:M], topk_weights=w[:M])
    torch.cuda.synchronize()
    assert (ids[M:] == -7).all() and (w[M:] == -7.0).all()
    return ids[:M].cpu().numpy(), w[:M].cpu().numpy().astype(np.float64)


def check(l, k, score="softmax", renorm=True, bias=None, G=1, kept=1, top=1, scale=1.0):
    moe = _moe()
    r = moe.Routing(k, score=score, renormalize=renorm,
                    select_bias=None if bias is None else h.dev_f32(bias), n_group=G,
                    topk_group=kept, group_top=top, scale=scale)
    ids, w = run_select(l, r)
    ref = mo.select_ids(l, k, score, bias, G, kept, top)
    assert np.array_equal(ids, ref)
    wr = mo.select_weights(l, ref, score, renorm, scale)
    # fp32 has nothing below 2^-149; products with scale flush there
    assert np.all(np.abs(w - wr) <= rel_tol(l, k) * np.abs(wr) + 2.0 ** -126 * max(1.0, abs(scale)))
    return ids, w


RULES = [
    # E, k, score, renorm, bias, n_group, topk_group, group_top
    (256, 8, "sigmoid", True, True, 8, 4, 2),
    (256, 8, "sigmoid", True, False, 8, 4, 2),
    (256, 8, "softmax", False, True, 8, 4, 1),
    (160, 6, "softmax", False, False, 8, 3, 1),
    (128, 8, "softmax", True, False, 1, 1, 1),
    (128, 8, "softmax", True, True, 1, 1, 1),
    (60, 4, "softmax", False, True, 1, 1, 1),
    (60, 4, "sigmoid", False, True, 5, 2, 2),
    (512, 32, "sigmoid", True, True, 16, 5, 2),
    (512, 10, "sigmoid", True, True, 1, 1, 1),
    (512, 32, "softmax", True, False, 1, 1, 1),
    (510, 7, "softmax", True, True, 10, 3, 2),
    (64, 2, "sigmoid", True, True, 64, 9, 1),
    (48, 6, "sigmoid", True, True, 3, 2, 2),
    (33, 33 - 1, "sigmoid", True, True, 1, 1, 1),
    (7, 7, "softmax", True, True, 1, 1, 1),
    (12, 12, "sigmoid", True, True, 4, 4, 2),
    (2, 1, "softmax", False, True, 2, 1, 1),
    (1, 1, "sigmoid", False, False, 1, 1, 1),
    (1, 1, "softmax", True, True, 1, 1, 1),
]


@pytest.mark.parametrize("M", [1, 2, 5, 66])
@pytest.mark.parametrize("E,k,score,renorm,bias,G,kept,top", RULES)
def test_rules(E, k, score, renorm, bias, G, kept, top, M):
    l = draw(M, E, 100 * E + M + k)
    check(l, k, score, renorm, steps(E, E + k) if bias else None, G, kept, top, 2.5)


@pytest.mark.parametrize("seed", range(40))
def test_random_rules(seed):
    rng = np.random.default_rng(seed)
    G = int(rng.choice([1, 1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 20]))
    size = int(rng.integers(1, 512 // G + 1))
    E = G * size
    kept = int(rng.integers(1, G + 1))
    k = int(rng.integers(1, min(kept * size, 32) + 1))
    top = int(rng.integers(1, 3)) if G > 1 and size > 1 else 1
    l = draw(int(rng.integers(1, 90)), E, seed + 1000, float(rng.choice([0.3, 1.0, 6.0])))
    check(l, k, str(rng.choice(["softmax", "sigmoid"])), bool(rng.integers(2)),
          steps(E, seed) if rng.integers(2) else None, G, kept, top,
          float(rng.choice([1.0, 2.5, -0.5, 0.0])))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,kept,top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
@pytest.mark.parametrize("E", [64, 128, 256, 512])
def test_many_exact_ties(E, G, kept, top, score):
    """Few different logits and biases: most choices are ties, which go to
    the lower id and the lower group."""
    rng = np.random.default_rng(E + G)
    l = rng.integers(-1, 2, size=(40, E)).astype(np.float32)
    l[0] = 0.0
    l[1, : E // 2] = 1.0
    check(l, 8, score, True, None, G, kept, top)
    check(l, 8, score, True, np.zeros(E, np.float32), G, kept, top)
    check(l, 8, score, True, (rng.integers(-1, 2, size=E) * 0.25).astype(np.float32), G, kept, top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choices_one_rounding_apart(score):
    """Scores that fp32 cannot tell apart and 64 bits can: logits one fp32
    step apart, and biases that pull sums together."""
    M, E, k = 64, 256, 8
    rng = np.random.default_rng(8)
    base = draw(M, E, 77)
    l = base.copy()
    for t in range(M):
        order = np.argsort(-base[t])
        a, b = order[k - 1], order[k]
        l[t, b] = np.nextafter(l[t, a], np.float32(-9 if rng.integers(2) else 9))
    check(l, k, score)
    check(l, k, score, bias=np.zeros(E, np.float32))
    check(l, k, score, bias=steps(E, 4))
    # a bias that nearly undoes the score's difference of two experts
    s = np.exp(mo.log_scores(l[:1], score))[0]
    order = np.argsort(-s)
    b = np.zeros(E, dtype=np.float32)
    b[order[k]] = np.float32(s[order[k - 1]] - s[order[k]])
    for off in (-1, 0, 1):
        c = b.copy()
        if off:
            c[order[k]] = np.nextafter(c[order[k]], np.float32(off))
        check(l[:1], k, score, bias=c)
        check(l[:1], k, score, bias=c, G=4, kept=2, top=2)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts(score, renorm):
    """-inf logits: some, all but one, all but fewer than top_k, every one."""
    E, k = 128, 6
    l = draw(9, E, 3)
    l[1, ::2] = -INF
    l[2, 1:] = -INF
    l[3, 4:] = -INF
    l[4, :] = -INF
    l[5, :] = np.finfo(np.float32).min
    l[6, 5:] = np.finfo(np.float32).min
    for bias in (None, np.zeros(E, np.float32)):
        check(l, k, score, renorm, bias)
        check(l, k, score, renorm, bias, 8, 3, 1)
        check(l, k, score, renorm, bias, 8, 3, 2)
    # a bias of -inf puts an expert behind all others
    b = np.zeros(E, dtype=np.float32)
    b[::3] = -INF
    ids, _ = check(l[:1], k, score, renorm, b)
    assert np.all(ids % 3 != 0)
    b[:] = -INF
    b[100] = 0.0
    check(l, k, score, renorm, b)


def test_underflowing_scores_renormalize_exactly():
    l = np.full((3, 64), -1000.0, dtype=np.float32)
    l[0, 5], l[0, 9] = -900.0, -901.0
    l[1] -= np.arange(64)
    l[2] = -88.0 - np.arange(64) / 4
    for score in ("sigmoid", "softmax"):
        _, w = check(l, 4, score)
        assert np.allclose(w.sum(1), 1.0, atol=1e-6)


def test_not_a_number_stays_in_its_row():
    """NaN and +inf rows give distinct ids in range and disturb no other row."""
    moe = _moe()
    l = draw(8, 96, 21)
    bad = l.copy()
    bad[1, 3] = np.nan
    bad[3, :] = np.nan
    bad[5, 7] = INF
    b = steps(96, 2)
    for score in ("softmax", "sigmoid"):
        for bias in (None, b):
            for G in (1, 4):
                r = moe.Routing(5, score=score, select_bias=None if bias is None else h.dev_f32(bias),
                                n_group=G, topk_group=min(G, 2), group_top=1)
                ids, w = run_select(bad, r)
                good_ids, good_w = run_select(l, r)
                keep = [0, 2, 4, 6, 7]
                assert np.array_equal(ids[keep], good_ids[keep])
                assert np.array_equal(w[keep], good_w[keep])
                assert np.all((ids >= 0) & (ids < 96))
                assert all(len(set(row)) == 5 for row in ids.tolist())
                if score == "sigmoid":
                    # a NaN ranks behind every number, a +inf before
                    assert not np.any(ids[1] == 3) and np.all(np.isfinite(w[1]))
                    if bias is None:
                        assert ids[5, 0] == 7


def test_largest_sizes():
    check(draw(4099, 512, 5), 32, "sigmoid", True, steps(512, 5), 8, 3, 2)
    check(draw(16385, 60, 6), 4, "softmax", False)


def test_bias_is_read_at_each_call():
    import torch
    moe = _moe()
    l = draw(20, 64, 2)
    b = h.dev_f32(np.zeros(64))
    r = moe.Routing(4, score="sigmoid", select_bias=b)
    ids0, _ = run_select(l, r)
    b[17] = 2.0
    ids1, _ = run_select(l, r)
    torch.cuda.synchronize()
    assert not np.all(ids0[:, 0] == 17) and np.all(ids1[:, 0] == 17)


# ---------------------------------------------------------------------------
# the gradient
# ---------------------------------------------------------------------------

def run_backward(l, ids, g, routing, tail=2):
    import torch
    moe = _moe()
    M, E = l.shape
    out = torch.full((M + tail, E), -7.0, dtype=torch.float32, device="cuda")
    dst = out[:M]
    moe.moe_select_backward(h.dev_f32(l), h.dev_i32(ids), h.dev_f32(g), routing, grad_logits=dst)
    torch.cuda.synchronize()
    assert (out[M:] == -7.0).all()
    return dst.cpu().numpy().astype(np.float64)


def check_backward(l, ids, score, renorm, scale, seed):
    moe = _moe()
    M, k = ids.shape
    g = draw(M, k, seed)
    got = run_backward(l, ids, g, moe.Routing(k, score=score, renormalize=renorm, scale=scale))
    ref = mo.select_backward(l, ids, g, score, renorm, scale)
    # every term is a product of factors <= 1 with scale * g: errors of the
    # weights (rel_tol each) and of sums of k terms
    tol = (3 * rel_tol(l, k) + 2 * k * 2.0 ** -23) * abs(scale) * np.abs(g).sum(1, keepdims=True)
    assert np.all(np.abs(got - ref) <= tol + 2.0 ** -126)
    return got, g


@pytest.mark.parametrize("M", [1, 3, 66])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(256, 8), (128, 8), (60, 4), (512, 32), (512, 1), (33, 5), (7, 7),
                                 (1, 1), (130, 2)])
def test_backward(E, k, score, renorm, M):
    l = draw(M, E, E + k + M, 1.5)
    check_backward(l, mo.select_ids(l, k, score), score, renorm, 2.5, 5)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_backward_against_differences(score, renorm):
    """The kernel's gradient against central differences of the float64
    weights (error of the quotient below 1e-8)."""
    M, E, k, eps = 2, 12, 3, 1e-5
    l = draw(M, E, 31)
    ids = mo.select_ids(l, k, score)
    got, g = check_backward(l, ids, score, renorm, 1.0, 6)

    def loss(v):
        p = np.exp(mo.log_scores(v, score))
        s = np.take_along_axis(p, ids.astype(np.int64), axis=1)
        return float(((s / s.sum(1, keepdims=True) if renorm else s) * g).sum())

    for t in range(M):
        for e in range(E):
            up, down = l.astype(np.float64), l.astype(np.float64)
            up[t, e] += eps
            down[t, e] -= eps
            fd = (loss(up) - loss(down)) / (2 * eps)
            assert abs(fd - got[t, e]) <= 1e-8 + (3 * rel_tol(l, k)) * np.abs(g[t]).sum()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_backward_masked_rows_and_odd_ids(score, renorm):
    E, k = 96, 4
    l = draw(6, E, 41)
    l[1, ::2] = -INF
    l[2, 2:] = -INF
    l[3, :] = -INF
    l[4, :] = -1000.0
    ids = mo.select_ids(l, k, score)
    got, g = check_backward(l, ids, score, renorm, 1.0, 7)
    assert np.all(got[3] == 0.0)
    # the same id twice: both slots' gradients; an id out of range: no part
    ids2 = ids.copy()
    ids2[0] = [5, 9, 5, 5]
    check_backward(l, ids2, score, renorm, 1.0, 8)
    ids3 = ids.copy()
    ids3[0, 1], ids3[5, 2] = -1, E
    moe = _moe()
    got3 = run_backward(l, ids3, g, moe.Routing(k, score=score, renormalize=renorm))
    for t, keep in ((0, [0, 2, 3]), (5, [0, 1, 3])):
        ref = mo.select_backward(l[t:t + 1], ids3[t:t + 1][:, keep], g[t:t + 1][:, keep], score,
                                 renorm, 1.0)
        tol = (3 * rel_tol(l[t:t + 1], k) + 8 * 2.0 ** -23) * np.abs(g[t]).sum()
        assert np.abs(got3[t] - ref[0]).max() <= tol


def test_backward_large_and_repeatable():
    l = draw(8193, 512, 51)
    moe = _moe()
    ids, _ = run_select(l, moe.Routing(10, score="sigmoid"))
    r = moe.Routing(10, score="sigmoid", scale=2.5)
    g = draw(8193, 10, 52)
    a = run_backward(l, ids, g, r)
    b = run_backward(l, ids, g, r)
    assert np.array_equal(a, b)
    ref = mo.select_backward(l[-40:], ids[-40:], g[-40:], "sigmoid", True, 2.5)
    tol = (3 * rel_tol(l, 10) + 20 * 2.0 ** -23) * 2.5 * np.abs(g[-40:]).sum(1, keepdims=True)
    assert np.all(np.abs(a[-40:] - ref) <= tol)


# ---------------------------------------------------------------------------
# through the router, and in a user's program
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M", [1, 17, 300])
def test_route_scored(M):
    import torch
    moe = _moe()
    lay = wl.make_layer("qwen15", M, I=8)
    d = h.layer_to_device(lay)
    b = steps(60, 3)
    r = moe.Routing(4, score="sigmoid", select_bias=h.dev_f32(b), n_group=4, topk_group=2,
                    group_top=2, scale=1.5)
    logits = torch.empty((M, 60), dtype=torch.float32, device="cuda")
    ids, w = moe.moe_route_scored(d["x"], d["w_router"], r, logits_out=logits)
    ids2, w2 = moe.moe_route_scored(d["x"], d["w_router"], r)
    torch.cuda.synchronize()
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    l = logits.cpu().numpy()
    assert np.abs(l - mo.router_logits(lay["x"], lay["w_router"])).max() < 1e-4
    ref = mo.select_ids(l, 4, "sigmoid", b, 4, 2, 2)
    assert np.array_equal(ids.cpu().numpy(), ref)
    wr = mo.select_weights(l, ref, "sigmoid", True, 1.5)
    assert np.abs(w.cpu().numpy() - wr).max() <= rel_tol(l, 4) * 1.5


def test_select_captured_and_on_two_streams():
    """Two captured calls replayed between eager ones, and two streams at
    once: every result is the eager one's, bit for bit."""
    import torch
    moe = _moe()
    ls = [h.dev_f32(draw(700, 256, 60 + i)) for i in range(2)]
    bias = h.dev_f32(steps(256, 9))
    r = moe.Routing(8, score="sigmoid", select_bias=bias, n_group=8, topk_group=4, group_top=2)
    gw = h.dev_f32(draw(700, 8, 66))

    def step(l, stream=None):
        ids, w = moe.moe_select(l, r, stream=stream)
        return ids, w, moe.moe_select_backward(l, ids, gw, r, stream=stream)

    want = [step(l) for l in ls]
    torch.cuda.synchronize()
    graphs = []
    for l in ls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step(l)
        graphs.append((g, got))
    for _ in range(3):
        for (g, got), exp in zip(graphs, want):
            g.replay()
            eager = step(ls[0])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, exp))
            assert all(torch.equal(a, b) for a, b in zip(eager, want[0]))
    streams = [torch.cuda.Stream() for _ in ls]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    out = [[step(l, s) for l, s in zip(ls, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for rnd in out:
        for got, exp in zip(rnd, want):
            assert all(torch.equal(a, b) for a, b in zip(got, exp))


def test_binding_refuses_wrong_tensors():
    import torch
    moe = _moe()
    l = h.dev_f32(draw(6, 64, 1))
    r = moe.Routing(4)
    ids, w = moe.moe_select(l, r)
    for bad in (l.double(), l.half(), l.t(), l[:, ::2]):
        with pytest.raises(ValueError):
            moe.moe_select(bad, r)
    with pytest.raises(ValueError):
        moe.moe_select(l, r, topk_ids=ids.long())
    with pytest.raises(ValueError):
        moe.moe_select(l, r, topk_weights=w[:3])
    with pytest.raises(ValueError):
        moe.moe_select(l, moe.Routing(4, select_bias=h.dev_f32(np.zeros(63))))
    with pytest.raises(ValueError):
        moe.moe_select_backward(l, ids, w[:, :2], r)
    with pytest.raises(moe.MoeError):
        moe.moe_select(l, moe.Routing(65))
    with pytest.raises(moe.MoeError):
        moe.moe_select_backward(l, ids, w, r, grad_logits=l)
    with pytest.raises(moe.MoeError):
        moe.moe_select(l, moe.Routing(4, n_group=5))
    empty = moe.moe_select(l[:0], r)
    assert empty[0].shape == (0, 4) and empty[1].shape == (0, 4)
