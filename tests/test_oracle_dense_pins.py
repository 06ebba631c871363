"""The float64 oracle of the dense operators against torch's autograd in
float64, differences and values known by hand."""

from __future__ import annotations

import math

import numpy as np
import torch

from oracle import dense_oracle as do


def test_token_logprobs_by_hand():
    l = np.log(np.array([[0.5, 0.25, 0.125, 0.125]])) + 7.0
    r = do.token_logprobs(l, np.array([2]), 4)
    assert abs(r["logprobs"][0] - math.log(0.125)) < 1e-12
    assert abs(r["entropy"][0] - 1.75 * math.log(2)) < 1e-12
    assert abs(r["lse"][0] - 7.0) < 1e-12
    assert r["top_ids"].tolist() == [[0, 1, 2, 3]]
    assert np.allclose(r["top_logprobs"], np.log([[0.5, 0.25, 0.125, 0.125]]))


def test_token_logprobs_rows_that_are_not_finite():
    inf = np.inf
    l = np.array([[-inf, -inf, -inf], [0.0, -inf, 0.0], [np.nan, 1.0, -inf], [inf, 1.0, -inf]])
    r = do.token_logprobs(l, np.array([1, 1, 0, -1]), 3)
    assert r["lse"][0] == -inf and r["entropy"][0] == 0 and r["logprobs"][0] == -inf
    assert r["top_ids"][0].tolist() == [0, 1, 2]
    assert r["logprobs"][1] == -inf and abs(r["entropy"][1] - math.log(2)) < 1e-12
    assert r["top_ids"][1].tolist() == [0, 2, 1]
    assert np.isnan([r["lse"][2], r["entropy"][2], r["logprobs"][2]]).all()
    assert r["top_ids"][2].tolist() == [1, 2, 0]
    assert r["logprobs"][3] == 0 and r["top_ids"][3].tolist() == [0, 1, 2]


def test_token_logprobs_and_gradient_against_autograd():
    g = torch.Generator().manual_seed(3)
    l = (torch.randn((5, 40), generator=g, dtype=torch.float64) * 3).requires_grad_()
    tok = torch.randint(0, 40, (5,), generator=g)
    a, b = torch.randn((2, 5), generator=g, dtype=torch.float64)
    logp = torch.log_softmax(l, dim=1)
    lp, ent = logp.gather(1, tok[:, None])[:, 0], -(logp.exp() * logp).sum(1)
    (lp * a + ent * b).sum().backward()
    r = do.token_logprobs(l.detach().numpy(), tok.numpy(), 4)
    assert np.allclose(r["logprobs"], lp.detach().numpy(), atol=1e-12)
    assert np.allclose(r["entropy"], ent.detach().numpy(), atol=1e-12)
    assert np.array_equal(r["top_ids"], torch.topk(l, 4)[1].numpy())
    d = do.token_logprobs_backward(l.detach().numpy(), tok.numpy(), r["lse"], r["entropy"],
                                   a.numpy(), b.numpy())
    assert np.allclose(d, l.grad.numpy(), atol=1e-12)


def test_token_logprobs_gradient_of_rows_ruled_out():
    l = np.full((2, 3), -np.inf)
    l[1, 1] = 2.0
    r = do.token_logprobs(l, np.array([0, -1]))
    with np.errstate(invalid="ignore"):
        d = do.token_logprobs_backward(l, np.array([0, -1]), r["lse"], r["entropy"], np.ones(2),
                                       np.ones(2))
    assert not d.any()      # nothing to choose, and one certain token that is not asked for


def test_gated_against_autograd():
    g = torch.Generator().manual_seed(4)
    x = torch.randn((6, 10), generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn((14, 10), generator=g, dtype=torch.float64, requires_grad=True)
    d = torch.randn((6, 7), generator=g, dtype=torch.float64)
    y = torch.nn.functional.silu(x @ w[:7].T) * (x @ w[7:].T)
    (y * d).sum().backward()
    assert np.allclose(do.gated(x.detach().numpy(), w.detach().numpy()), y.detach().numpy(), atol=1e-12)
    gx, gw = do.gated_backward(x.detach().numpy(), w.detach().numpy(), d.numpy())
    assert np.allclose(gx, x.grad.numpy(), atol=1e-12) and np.allclose(gw, w.grad.numpy(), atol=1e-12)


def test_adapters_against_merged_weights():
    rng = np.random.default_rng(5)
    x, a, b = rng.standard_normal((9, 8)), rng.standard_normal((3, 4, 8)), rng.standard_normal((3, 6, 4))
    sc, add = rng.random(3), rng.standard_normal((9, 6))
    slots = np.array([0, 1, 2, -1, 3, 1, 0, 2, 2])
    y = do.adapters(x, a, b, sc, slots, add)
    for m, s in enumerate(slots):
        w = sc[s] * b[s] @ a[s] if 0 <= s < 3 else np.zeros((6, 8))
        assert np.allclose(y[m], add[m] + w @ x[m])
    z = do.adapters(x, a, b, None, slots, add, True)
    y = do.adapters(x, a, b, np.ones(3), slots, add)
    assert np.allclose(z, y[:, :3] / (1 + np.exp(-y[:, :3])) * y[:, 3:])
