"""The bf16 gated block on the GPU (moe_linear_gated and its gradient) against
the float64 oracle."""

from __future__ import annotations

import numpy as np
import pytest

import moe_workloads as wl
from oracle import dense_oracle as do
from oracle import moe_oracle as mo
from tests import helpers as h

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
B = 2.0 ** -8      # half a bf16 step, relative


def _moe():
    import mixture_experts_ffn_renorm_amd as moe
    return moe


def bits(a):
    return wl.f32_to_bf16_bits(np.asarray(a, dtype=np.float32))


def inputs(M, H, I, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    x = bits(rng.standard_normal((M, H)))
    w = bits(rng.standard_normal((2 * I, H)) * spread / np.sqrt(H))
    d = bits(rng.standard_normal((M, I)))
    return x, w, d


def parts(x, w):
    """gate and up in float64 and bounds of their fp32 errors: H exact products
    of size sum |x||w|, at most H / 16 + 64 roundings in a row."""
    X, W = mo.widen_bf16(x).astype(np.float64), mo.widen_bf16(w).astype(np.float64)
    I = W.shape[0] // 2
    y, e = X @ W.T, (X.shape[1] / 16 + 64) * U * (np.abs(X) @ np.abs(W).T)
    return X, W, y[:, :I], y[:, I:], e[:, :I], e[:, I:]


def act_bound(g, u, eg, eu):
    """|SiLU'| <= 1.1; the fast exponential's argument rounds by |g| 2^-23, it
    and the quotient by a few units; then one bf16 rounding."""
    s = 1 / (1 + np.exp(-g))
    act = np.abs(g * s)
    e = 1.1 * eg * np.abs(u) + act * eu + 1.1 * eg * eu + act * np.abs(u) * (np.abs(g) + 8) * 2 * U
    return e + (act * np.abs(u) + e) * B + 2.0 ** -133


def check(M, H, I, seed=0, data=None):
    import torch
    moe = _moe()
    x, w, _ = inputs(M, H, I, seed) if data is None else data
    buf = torch.full((M * I + 64,), -7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:M * I].view(M, I)
    assert moe.moe_linear_gated(h.dev_bf16(x), h.dev_bf16(w), out=out) is out
    torch.cuda.synchronize()
    assert (buf[M * I:] == -7.0).all()
    X, W, g, u, eg, eu = parts(x, w)
    err = np.abs(h.host_bf16_to_f64(out) - do.gated(X, W))
    bound = act_bound(g, u, eg, eu)
    assert np.all(err <= bound), (err / bound).max()
    return out


MS = [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 257, 300,
      512, 600]


@pytest.mark.parametrize("M", MS)
def test_batches(M):
    check(M, 256, 136, M)


@pytest.mark.parametrize("M", [1, 3, 12, 40, 150])
@pytest.mark.parametrize("H", [8, 16, 24, 32, 40, 56, 64, 72, 120, 128, 136, 248, 504, 1408, 2040,
                               2048, 5632, 8200])
def test_inner_sizes(H, M):
    check(M, H, 40, H)


@pytest.mark.parametrize("M", [1, 6, 50, 140])
@pytest.mark.parametrize("I", [8, 16, 24, 56, 64, 72, 128, 136, 264, 1000, 1408])
def test_output_sizes(I, M):
    check(M, 192, I, I)


@pytest.mark.parametrize("M,H,I", [(1, 2048, 5632), (64, 2048, 5632), (509, 2048, 1408),
                                   (2100, 256, 1500), (4100, 64, 520), (2100, 64, 4096)])
def test_layer_sizes(M, H, I):
    # (I multiple of 8)
    check(M, H, I // 8 * 8, 3)


@pytest.mark.parametrize("M", [4, 5, 16, 17, 32, 33, 64, 65, 128])
@pytest.mark.parametrize("H,I", [(264, 8200), (136, 16648)])
def test_few_rows_of_many_features(H, I, M):
    check(M, H, I, M)


@pytest.mark.parametrize("M", [2, 20, 70, 300])
def test_a_row_that_is_not_finite_stays_alone(M):
    import torch
    moe = _moe()
    x, w, _ = inputs(M, 200, 72, 5)
    x, w = h.dev_bf16(x), h.dev_bf16(w)
    good = moe.moe_linear_gated(x, w)
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[M - 1, 199] = bad
        out = moe.moe_linear_gated(y, w)
        torch.cuda.synchronize()
        assert not torch.isfinite(out[M - 1]).any() or bad == float("inf")
        assert torch.equal(out[:M - 1], good[:M - 1])


def test_large_gates():
    """Gates far from 0 on both sides: SiLU(g) = g or 0, no overflow."""
    x, w, d = inputs(70, 64, 40, 6, spread=60.0)
    check(70, 64, 40, data=(x, w, d))
    check(3, 64, 40, data=(x[:3], w, d[:3]))
    check_grad(70, 64, 40, data=(x, w, d))


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------

def grad_bounds(x, w, d, rounding=B):
    """Bounds of grad_x and grad_w13: the errors of d_gate and d_up (those of
    gate and up through derivatives of at most 1.1, and SiLU's second
    derivative, at most 0.5; a few fp32 roundings; one rounding more), then
    fp32 sums, then one bf16 rounding."""
    X, W, g, u, eg, eu = parts(x, w)
    D = mo.widen_bf16(d).astype(np.float64)
    s = 1 / (1 + np.exp(-g))
    ds = s * (1 + g * (1 - s))
    dg, du = D * u * ds, D * g * s
    few = (np.abs(g) + 12) * 2 * U
    edg = np.abs(D) * (1.1 * eu + np.abs(u) * (0.5 * eg + few * s * (1 + np.abs(g))))
    edu = np.abs(D) * (1.1 * eg + np.abs(g) * s * few)
    edg += (np.abs(dg) + edg) * rounding + 2.0 ** -133
    edu += (np.abs(du) + edu) * rounding + 2.0 ** -133
    v, ev = np.concatenate([dg, du], 1), np.concatenate([edg, edu], 1)

    def product(a, ea, b, K):
        ref = a @ b
        e = ea @ np.abs(b) + (K / 16 + 80) * U * ((np.abs(a) + ea) @ np.abs(b))
        return ref, e + (np.abs(ref) + e) * B + 2.0 ** -133

    return product(v, ev, W, v.shape[1]), product(v.T, ev.T, X, v.shape[0])


def check_grad(M, H, I, seed=0, data=None, need=(True, True)):
    import torch
    moe = _moe()
    x, w, d = inputs(M, H, I, seed) if data is None else data
    ws = torch.full((moe.moe_linear_gated_backward_workspace_size(M, H, I) + 64,), 255,
                    dtype=torch.uint8, device="cuda")      # NaN everywhere
    bufs, outs = [], []
    for rows, wanted in ((M, need[0]), (2 * I, need[1])):
        b = torch.full((rows * H + 64,), -7.0, dtype=torch.bfloat16, device="cuda")
        bufs.append(b)
        outs.append(b[:rows * H].view(rows, H) if wanted else None)
    got = moe.moe_linear_gated_backward(h.dev_bf16(x), h.dev_bf16(w), h.dev_bf16(d),
                                        grad_x=outs[0], grad_w13=outs[1], need_x=need[0],
                                        need_w13=need[1], ws=ws[:-64])
    torch.cuda.synchronize()
    assert (ws[-64:] == 255).all()
    # 16 rows or fewer: d_gate and d_up are two bf16 numbers each, off by 2^-8 of 2^-8
    ref = do.gated_backward(*(mo.widen_bf16(t).astype(np.float64) for t in (x, w, d)))
    bounds = grad_bounds(x, w, d, B * B if M <= 16 else B)
    for b, out, g, wanted, (_, bound), want in zip(bufs, outs, got, need, bounds, ref):
        if not wanted:
            assert g is None and (b == -7.0).all()
            continue
        assert g is out and (b[-64:] == -7.0).all()
        err = np.abs(h.host_bf16_to_f64(g) - want)
        assert np.all(err <= bound), (err / bound).max()
    return got


@pytest.mark.parametrize("M", MS)
def test_gradient_batches(M):
    check_grad(M, 136, 72, M)


@pytest.mark.parametrize("M", [1, 33, 150])
@pytest.mark.parametrize("H,I", [(8, 8), (16, 24), (40, 8), (8, 264), (264, 72), (504, 136),
                                 (1000, 1000), (2048, 40), (64, 2048)])
def test_gradient_sizes(H, I, M):
    check_grad(M, H, I, H + I)


@pytest.mark.parametrize("M", [1, 2, 7, 15, 16])
@pytest.mark.parametrize("H,I", [(128, 64), (2048, 264), (40000, 72), (72, 4104)])
def test_gradient_of_the_fewest_rows(H, I, M):
    check_grad(M, H, I, 8)
    check_grad(M, H, I, 9, need=(M % 2 == 0, M % 2 == 1))


@pytest.mark.parametrize("M,H,I", [(7, 72, 8200), (31, 136, 8264), (60, 72, 16648),
                                   (200, 2048, 4096), (511, 2048, 4096), (513, 2048, 4096)])
def test_gradient_of_many_features(M, H, I):
    check_grad(M, H, I, 6)


@pytest.mark.parametrize("need", [(True, False), (False, True)])
@pytest.mark.parametrize("M", [5, 300])
def test_one_gradient_alone(M, need):
    check_grad(M, 264, 136, 4, need=need)


@pytest.mark.parametrize("M,H,I", [(509, 2048, 1408), (2100, 256, 1504), (4099, 512, 264),
                                   (40, 2048, 5632), (2100, 64, 4096), (2100, 8192, 8)])
def test_gradient_layer_sizes(M, H, I):
    check_grad(M, H, I, 9)


def test_gradient_against_differences():
    """Central differences of the definition, along random directions."""
    M, H, I = 37, 96, 40
    x, w, d = inputs(M, H, I, 12)
    gx, gw = (h.host_bf16_to_f64(t) for t in check_grad(M, H, I, data=(x, w, d)))
    X, W, D = (mo.widen_bf16(t).astype(np.float64) for t in (x, w, d))
    (_, bx), (_, bw) = grad_bounds(x, w, d)
    rng = np.random.default_rng(3)
    eps = 1e-5
    for _ in range(8):
        vx, vw = rng.standard_normal(X.shape), rng.standard_normal(W.shape)
        f = [(do.gated(X + t * eps * vx, W + t * eps * vw) * D).sum() for t in (1, -1)]
        diff = (f[0] - f[1]) / (2 * eps)
        mine = (gx * vx).sum() + (gw * vw).sum()
        # the kernel's bound along the direction; differences: eps^2 times a
        # third derivative, and cancellation of 2^-52 |f| / eps, are far below
        bound = (bx * np.abs(vx)).sum() + (bw * np.abs(vw)).sum()
        assert abs(diff - mine) <= bound + 1e-4 * abs(diff)


def test_no_rows():
    import torch
    moe = _moe()
    x, w, d = inputs(4, 64, 24, 1)
    x, w, d = h.dev_bf16(x), h.dev_bf16(w), h.dev_bf16(d)
    assert moe.moe_linear_gated(x[:0], w).shape == (0, 24)
    g = torch.full((48, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    gx, gw = moe.moe_linear_gated_backward(x[:0], w, d[:0], grad_w13=g)
    assert gx.shape == (0, 64) and gw is g and not g.any()


# ---------------------------------------------------------------------------
# streams, graphs, refusals
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M", [1, 48, 300])
def test_repeatable_captured_and_on_two_streams(M):
    import torch
    moe = _moe()
    data = [[h.dev_bf16(t) for t in inputs(M, 512, 264, 20 + i)] for i in range(2)]

    def both(x, w, d, stream=None):
        return (moe.moe_linear_gated(x, w, stream=stream),
                *moe.moe_linear_gated_backward(x, w, d, stream=stream))

    want = [both(*t) for t in data]
    torch.cuda.synchronize()
    graphs = []
    for t in data:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both(*t)
        graphs.append((g, out))
    for _ in range(3):
        for (g, out), exp in zip(graphs, want):
            for t in out:
                t.zero_()
            g.replay()
            again = both(*data[0])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, exp))
            assert all(torch.equal(a, b) for a, b in zip(again, want[0]))
    streams = [torch.cuda.Stream() for _ in data]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    out = [[both(*t, stream=s) for t, s in zip(data, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for rnd in out:
        for a, b in zip(rnd, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_a_workspace_serves_fewer_rows():
    import torch
    moe = _moe()
    for H, I in ((64, 40), (2048, 1408), (8192, 8)):
        sizes = [moe.moe_linear_gated_backward_workspace_size(M, H, I) for M in
                 (1, 5, 64, 128, 129, 500, 1000, 2048, 4096, 8192, 20000)]
        assert sizes == sorted(sizes)
    del torch


def test_binding_refuses_wrong_tensors():
    import torch
    moe = _moe()
    x, w, d = (h.dev_bf16(t) for t in inputs(6, 64, 24, 2))
    for bad in (x.float(), x.half(), x[:, ::2], x.t().contiguous().t()):
        with pytest.raises((ValueError, moe.MoeError)):
            moe.moe_linear_gated(bad, w)
        with pytest.raises((ValueError, moe.MoeError)):
            moe.moe_linear_gated_backward(bad, w, d)
    with pytest.raises(moe.MoeError):
        moe.moe_linear_gated(x, w[:47])
    with pytest.raises((ValueError, moe.MoeError)):
        moe.moe_linear_gated(x, w[:24])          # I = 12
    with pytest.raises(ValueError):
        moe.moe_linear_gated(x, w, out=d[:5])
    with pytest.raises(ValueError):
        moe.moe_linear_gated_backward(x, w, d[:, :16].contiguous())
    with pytest.raises(moe.MoeError):
        moe.moe_linear_gated_backward(x, w, d, need_x=False, need_w13=False)
    with pytest.raises(ValueError):
        moe.moe_linear_gated_backward(x, w, d, grad_x=torch.empty_like(x), need_x=False)
    with pytest.raises(moe.MoeError):
        moe.moe_linear_gated_backward(x, w, d, grad_x=x)
    with pytest.raises(moe.MoeError):
        moe.moe_linear_gated_backward(x, w, d, ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_linear_gated(x.cpu(), w)
