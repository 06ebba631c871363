"""Dense 4-bit products on the GPU (moe_linear_quantized) against the float64
oracle, and the layers with a routing rule that they stand beside."""

from __future__ import annotations

import numpy as np
import pytest

import moe_workloads as wl
from oracle import moe_oracle as mo
from tests import helpers as h

pytestmark = pytest.mark.gpu


def _moe():
    import mixture_experts_ffn_renorm_amd as moe
    return moe


def matrix(N, K, group, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 2 ** 32, size=(N, K // 8), dtype=np.uint64).astype(np.uint32)
    a = np.sqrt(3.0 / K) * spread
    ng = K // group
    s = wl.f32_to_bf16_bits((2 * a / 15 * (1 + 0.1 * rng.standard_normal((N, ng)))).astype(np.float32))
    b = wl.f32_to_bf16_bits((-a * (1 + 0.1 * rng.standard_normal((N, ng)))).astype(np.float32))
    return q, s, b


def rows(M, K, seed):
    return wl.f32_to_bf16_bits(np.random.default_rng(seed).standard_normal((M, K)).astype(np.float32))


def to_device(q, s, b, group):
    import torch
    return dict(bits=4, group_size=group,
                q=torch.from_numpy(q.view(np.int32).copy()).cuda(), scales=h.dev_bf16(s),
                biases=h.dev_bf16(b))


def error_bound(x, q, s, b, group, gated, row_scale, addend):
    """Bound of |out - exact| for fp32 accumulation of exact products: a dot
    of K terms of the size T = sum |x| (143 |s| + 128 |s| + |b|) (codes are
    multiplied as 128 + q and the 128 taken off), at most K / 32 + 64
    roundings of 2^-24 in a row; the epilogue's few; one bf16 rounding."""
    X = np.abs(mo.widen_bf16(x))
    K = X.shape[1]
    G = X.reshape(X.shape[0], K // group, group).sum(2)
    T = G @ (271 * np.abs(mo.widen_bf16(s)) + np.abs(mo.widen_bf16(b))).T
    e = (K / 32 + 64) * 2.0 ** -24 * T
    y = mo.linear_quantized(x, q, s, b, group)
    if gated:
        n = y.shape[1] // 2
        g, u, eg, eu = y[:, :n], y[:, n:], e[:, :n], e[:, n:]
        act = np.abs(g / (1 + np.exp(-g)))
        # |SiLU'| <= 1.1; the fast exponential's argument rounds by |g| 2^-23
        e = 1.1 * eg * np.abs(u) + act * eu + 1.1 * eg * eu + \
            act * np.abs(u) * (np.abs(g) + 8) * 2.0 ** -22
        y = act * np.abs(u)
    y = np.abs(y) + e
    if row_scale is not None:
        r = np.abs(row_scale.astype(np.float64))[:, None]
        e, y = e * r + y * r * 2.0 ** -24, y * r
    if addend is not None:
        e = e + (y + np.abs(mo.widen_bf16(addend))) * 2.0 ** -24
    return e


def check(M, N, K, group, seed=0, gated=False, scaled=False, added=False, in_place=False, tail=2,
          x=None, mat=None):
    import torch
    moe = _moe()
    q, s, b = matrix(N, K, group, seed) if mat is None else mat
    x = rows(M, K, seed + 1) if x is None else x
    n_out = N // 2 if gated else N
    rng = np.random.default_rng(seed + 2)
    rs = rng.random(M).astype(np.float32) if scaled else None
    ad = rows(M, n_out, seed + 3) if added else None
    buf = torch.full((M * n_out + tail * 8,), -7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:M * n_out].view(M, n_out)
    addend = None
    if added:
        addend = h.dev_bf16(ad)
        if in_place:
            out.copy_(addend)
            addend = out
    moe.moe_linear_quantized(h.dev_bf16(x), to_device(q, s, b, group), gated=gated,
                             row_scale=None if rs is None else h.dev_f32(rs), addend=addend, out=out)
    torch.cuda.synchronize()
    assert (buf[M * n_out:] == -7.0).all()
    ref = mo.linear_quantized(x, q, s, b, group, gated, rs, ad)
    e = error_bound(x, q, s, b, group, gated, rs, ad)
    got = h.host_bf16_to_f64(out)
    bound = e + (np.abs(ref) + e) * 2.0 ** -8 + 2.0 ** -133
    worst = np.abs(got - ref) / bound
    assert np.all(np.abs(got - ref) <= bound), f"{worst.max():.3f} of the bound"
    return out


MS = [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 31, 33, 64, 65, 130]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", MS)
def test_batches(M, group):
    check(M, 96, 512, group, seed=M)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 6, 40])
@pytest.mark.parametrize("N", [1, 2, 3, 15, 16, 17, 63, 65, 129, 1000])
def test_output_sizes(N, M, group):
    check(M, N, 256, group, seed=N)


@pytest.mark.parametrize("M", [1, 4, 20, 100])
@pytest.mark.parametrize("K,group", [(32, 32), (64, 32), (96, 32), (64, 64), (128, 128), (192, 64),
                                     (1408, 64), (1408, 128), (2080, 32), (2048, 64), (5632, 128),
                                     (8256, 64), (16384, 128)])
def test_inner_sizes(K, group, M):
    check(M, 40, K, group, seed=K)


@pytest.mark.parametrize("M", [1, 5, 24, 70])
@pytest.mark.parametrize("gated,scaled,added,in_place", [
    (True, False, False, False), (False, True, False, False), (False, False, True, False),
    (False, True, True, False), (True, True, True, False), (False, True, True, True),
    (True, False, True, True)])
def test_epilogues(M, gated, scaled, added, in_place):
    for N, group in ((70, 32), (256, 64)):
        check(M, N, 384, group if group == 64 else 32, 9, gated, scaled, added, in_place)


@pytest.mark.parametrize("seed", range(30))
def test_random_shapes(seed):
    rng = np.random.default_rng(seed)
    group = int(rng.choice([32, 64, 128]))
    K = group * int(rng.integers(1, 24))
    gated = bool(rng.integers(2))
    N = int(rng.integers(1, 300)) * (2 if gated else 1)
    check(int(rng.integers(1, 150)), N, K, group, seed, gated, bool(rng.integers(2)),
          bool(rng.integers(2)), bool(rng.integers(2)))


@pytest.mark.parametrize("M", [1, 16, 48])
def test_extreme_codes_and_scales(M):
    """Every code at its ends, scales of both signs and zero, biases that cancel."""
    N, K, group = 64, 256, 64
    q, s, b = matrix(N, K, group, 3)
    q[0], q[1], q[2], q[3] = 0, 0xFFFFFFFF, 0xF0F0F0F0, 0x0F0F0F0F
    s[4:8] |= 0x8000
    s[8:12] = 0
    b[12:16] = 0
    b[16:20] = wl.f32_to_bf16_bits(-8.0 * wl.bf16_bits_to_f32(s[16:20]))
    x = rows(M, K, 4)
    x[0, :64] = 0
    check(M, N, K, group, mat=(q, s, b), x=x)


@pytest.mark.parametrize("M", [1, 3, 16, 40])
def test_a_row_that_is_not_finite_stays_alone(M):
    import torch
    moe = _moe()
    K, group = 512, 64
    w = to_device(*matrix(48, K, group, 5), group)
    x = h.dev_bf16(rows(M, K, 6))
    good = moe.moe_linear_quantized(x, w)
    y = x.clone()
    y[M - 1, 7] = float("nan")
    bad = moe.moe_linear_quantized(y, w)
    torch.cuda.synchronize()
    assert torch.isnan(bad[M - 1]).all()
    assert torch.equal(bad[:M - 1], good[:M - 1])


def test_large_products():
    """A prefill-sized product, checked on a sample of its rows and columns."""
    import torch
    moe = _moe()
    # the last: more gate and up tiles per workgroup than its LDS holds, an
    # odd number of K slices
    for M, N, K, group, gated in ((1, 65537, 512, 64, False), (520, 4096, 2048, 64, False),
                                  (300, 5632, 1408, 128, True), (7, 480002, 384, 128, True)):
        q, s, b = matrix(N, K, group, 7)
        x = rows(M, K, 8)
        out = moe.moe_linear_quantized(h.dev_bf16(x), to_device(q, s, b, group), gated=gated)
        n_out = N // 2 if gated else N
        rng = np.random.default_rng(1)
        r = np.unique(np.concatenate([[0, M - 1], rng.integers(0, M, 6)]))
        c = np.unique(np.concatenate([[0, n_out - 1], rng.integers(0, n_out, 200)]))
        pick = np.concatenate([c, c + n_out]) if gated else c
        ref = mo.linear_quantized(x[r], q[pick], s[pick], b[pick], group, gated)
        e = error_bound(x[r], q[pick], s[pick], b[pick], group, gated, None, None)
        got = h.host_bf16_to_f64(out)[np.ix_(r, c)]
        assert np.all(np.abs(got - ref) <= e + (np.abs(ref) + e) * 2.0 ** -8)


@pytest.mark.parametrize("M", [1, 16, 200])
def test_repeatable_captured_and_on_two_streams(M):
    import torch
    moe = _moe()
    K, N, group = 1024, 768, 64
    ws = [to_device(*matrix(N, K, group, 20 + i), group) for i in range(2)]
    x = h.dev_bf16(rows(M, K, 22))
    want = [moe.moe_linear_quantized(x, w, gated=True) for w in ws]
    torch.cuda.synchronize()
    graphs = []
    for w in ws:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = moe.moe_linear_quantized(x, w, gated=True)
        graphs.append((g, out))
    for _ in range(3):
        for (g, out), exp in zip(graphs, want):
            out.zero_()
            g.replay()
            again = moe.moe_linear_quantized(x, ws[0], gated=True)
            torch.cuda.synchronize()
            assert torch.equal(out, exp) and torch.equal(again, want[0])
    streams = [torch.cuda.Stream() for _ in ws]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    out = [[moe.moe_linear_quantized(x, w, gated=True, stream=s) for w, s in zip(ws, streams)]
           for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for rnd in out for a, b in zip(rnd, want))


def test_binding_refuses_wrong_tensors():
    import torch
    moe = _moe()
    w = to_device(*matrix(32, 128, 64, 1), 64)
    x = h.dev_bf16(rows(4, 128, 2))
    for bad in (x.float(), x.half(), x[:, ::2], h.dev_bf16(rows(128, 4, 2)).t()):
        with pytest.raises((ValueError, moe.MoeError)):
            moe.moe_linear_quantized(bad, w)
    with pytest.raises(ValueError):
        moe.moe_linear_quantized(x, dict(w, scales=w["scales"][:, :1]))
    with pytest.raises(ValueError):
        moe.moe_linear_quantized(x, dict(w, q=w["q"].float()))
    with pytest.raises(ValueError):
        moe.moe_linear_quantized(x, w, row_scale=h.dev_f32(np.ones(3)))
    with pytest.raises(ValueError):
        moe.moe_linear_quantized(x, w, addend=x)
    with pytest.raises(ValueError):
        moe.moe_linear_quantized(x, w, out=torch.empty((4, 31), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.moe_linear_quantized(x, to_device(*matrix(31, 128, 64, 1), 64), gated=True)
    assert moe.moe_linear_quantized(x[:0], w).shape == (0, 32)


# ---------------------------------------------------------------------------
# the layers with a routing rule
# ---------------------------------------------------------------------------

RULE = dict(score="sigmoid", n_group=4, topk_group=2, group_top=2, scale=1.5)


def routing(k, E, **kw):
    moe = _moe()
    b = (np.round(np.random.default_rng(5).standard_normal(E) * 30) * 1e-3).astype(np.float32)
    return moe.Routing(k, select_bias=h.dev_f32(b), **{**RULE, **kw}), b


def check_layer(lay, d, out, ids, w, b, w13, w2):
    """The choice against the oracle's on the device's own logits, the output
    against the oracle's layer on that choice."""
    import torch
    moe = _moe()
    M, E, k = lay["M"], lay["E"], lay["top_k"]
    logits = torch.empty((M, E), dtype=torch.float32, device="cuda")
    r, _ = routing(k, E)
    moe.moe_route_scored(d["x"], d["w_router"], r, logits_out=logits)
    torch.cuda.synchronize()
    l = logits.cpu().numpy()
    ref = mo.select_ids(l, k, "sigmoid", b, 4, 2, 2)
    assert np.array_equal(ids.cpu().numpy(), ref)
    wr = mo.select_weights(l, ref, "sigmoid", True, 1.5)
    assert np.abs(w.cpu().numpy() - wr).max() <= 1e-5
    toks = h.sample_tokens(M, 12, 3)
    return toks, ref, wr


@pytest.mark.parametrize("M", [1, 3, 24, 300])
def test_forward_scored(M):
    import torch
    moe = _moe()
    lay = wl.make_layer("wide256", M, E=64, top_k=4, H=256, I=128)
    d = h.layer_to_device(lay)
    r, b = routing(4, 64)
    ids = torch.empty((M, 4), dtype=torch.int32, device="cuda")
    w = torch.empty((M, 4), dtype=torch.float32, device="cuda")
    out, info = moe.moe_forward_scored(d["x"], d["w_router"], d["w13"], d["w2"], r,
                                       topk_ids_out=ids, topk_weights_out=w)
    toks, ref, wr = check_layer(lay, d, out, ids, w, b, None, None)
    y = mo.layer_forward(lay["x"], lay["w13"], lay["w2"], ref, wr, toks)
    h.assert_close_outputs(h.host_bf16_to_f64(out)[toks], y)
    # the softmax rule through the scored call is the plain layer
    soft = moe.Routing(4)
    a, _ = moe.moe_forward_scored(d["x"], d["w_router"], d["w13"], d["w2"], soft, topk_ids_out=ids)
    ids2 = torch.empty_like(ids)
    c, _ = moe.moe_forward(d["x"], d["w_router"], d["w13"], d["w2"], 4, topk_ids_out=ids2)
    torch.cuda.synchronize()
    assert torch.equal(ids, ids2)
    h.assert_close_outputs(h.host_bf16_to_f64(a), h.host_bf16_to_f64(c))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [1, 24, 300])
def test_forward_quantized_scored(M, bits):
    import torch
    moe = _moe()
    lay = wl.make_quantized_layer("wide256", M, bits, E=64, top_k=4, H=256, I=128)
    d = dict(x=h.dev_bf16(lay["x"]), w_router=h.dev_bf16(lay["w_router"]))
    qw = dict(bits=bits)
    for n in ("w13", "w2"):
        qw[n + "_q"] = torch.from_numpy(lay[n + "_q"].view(np.int32).copy()).cuda()
        qw[n + "_scales"], qw[n + "_biases"] = h.dev_bf16(lay[n + "_scales"]), h.dev_bf16(
            lay[n + "_biases"])
    r, b = routing(4, 64)
    ids = torch.empty((M, 4), dtype=torch.int32, device="cuda")
    w = torch.empty((M, 4), dtype=torch.float32, device="cuda")
    out, info = moe.moe_forward_quantized_scored(d["x"], d["w_router"], qw, r, topk_ids_out=ids,
                                                 topk_weights_out=w)
    toks, ref, wr = check_layer(lay, d, out, ids, w, b, None, None)
    w13, w2 = mo.dequantized_experts(lay)
    h.assert_close_outputs(h.host_bf16_to_f64(out)[toks],
                           mo.layer_forward(lay["x"], w13, w2, ref, wr, toks))


@pytest.mark.parametrize("M", [1, 24, 300])
def test_forward_mxfp8_scored(M):
    import torch
    moe = _moe()
    lay = wl.make_mx_layer("wide256", M, E=64, top_k=4, H=256, I=128)
    d = dict(x=h.dev_bf16(lay["x"]), w_router=h.dev_bf16(lay["w_router"]))
    mxw = {n: torch.from_numpy(lay[n]).cuda() for n in
           ("w13_codes", "w13_scales", "w2_codes", "w2_scales")}
    r, b = routing(4, 64)
    ids = torch.empty((M, 4), dtype=torch.int32, device="cuda")
    w = torch.empty((M, 4), dtype=torch.float32, device="cuda")
    out, info = moe.moe_forward_mxfp8_scored(d["x"], d["w_router"], mxw, r, topk_ids_out=ids,
                                             topk_weights_out=w)
    toks, ref, wr = check_layer(lay, d, out, ids, w, b, None, None)
    full_ids, full_w = h.scatter_routing(M, toks, ref[toks], wr[toks])
    y = mo.mx_layer_forward(lay, full_ids, full_w, toks)[0]
    got = h.host_bf16_to_f64(out)[toks]
    h.assert_close_outputs(got, h.mx_boundary_reference(lay, full_ids, full_w, toks, got, y))


@pytest.mark.parametrize("M", [1, 20, 260])
def test_layer_with_a_shared_expert(M):
    """The operators together, as a quantized layer with a gated shared expert
    uses them: scored routing and experts, the shared expert's gate from a
    one-expert sigmoid rule, its two 4-bit products, the second added into
    the routed output; eagerly and replayed."""
    import torch
    moe = _moe()
    H, I, S, group = 256, 128, 320, 64
    lay = wl.make_quantized_layer("wide256", M, 4, E=64, top_k=4, H=H, I=I)
    x, wr_ = h.dev_bf16(lay["x"]), h.dev_bf16(lay["w_router"])
    qw = dict(bits=4)
    for n in ("w13", "w2"):
        qw[n + "_q"] = torch.from_numpy(lay[n + "_q"].view(np.int32).copy()).cuda()
        qw[n + "_scales"], qw[n + "_biases"] = h.dev_bf16(lay[n + "_scales"]), h.dev_bf16(
            lay[n + "_biases"])
    up, down = matrix(2 * S, H, group, 31), matrix(H, S, group, 32)
    dup, ddown = to_device(*up, group), to_device(*down, group)
    gate = rows(1, H, 33)
    gate_rule = moe.Routing(1, score="sigmoid", renormalize=False)
    r, b = routing(4, 64)
    ids = torch.empty((M, 4), dtype=torch.int32, device="cuda")
    w = torch.empty((M, 4), dtype=torch.float32, device="cuda")
    ws = moe.workspace(M, 64, 4, H, I)
    gws = torch.empty(max(16, 4 * M), dtype=torch.uint8, device="cuda")
    dgate = h.dev_bf16(gate)

    def step():
        y, _ = moe.moe_forward_quantized_scored(x, wr_, qw, r, topk_ids_out=ids, topk_weights_out=w,
                                                ws=ws)
        routed = y.clone()
        _, g = moe.moe_route_scored(x, dgate, gate_rule, ws=gws)
        act = moe.moe_linear_quantized(x, dup, gated=True)
        moe.moe_linear_quantized(act, ddown, row_scale=g.view(M), addend=y, out=y)
        return y, routed, g, act

    y, routed, g, act = step()
    torch.cuda.synchronize()
    check_layer(lay, dict(x=x, w_router=wr_), y, ids, w, b, None, None)
    gl = mo.router_logits(lay["x"], gate)
    assert np.abs(g.cpu().numpy() - 1 / (1 + np.exp(-gl))).max() < 1e-5
    abits = act.view(torch.int16).cpu().numpy().view(np.uint16)
    e = error_bound(lay["x"], *up, group, True, None, None)
    ra = mo.linear_quantized(lay["x"], *up, group, True)
    assert np.all(np.abs(h.host_bf16_to_f64(act) - ra) <= e + (np.abs(ra) + e) * 2.0 ** -8)
    rb = routed.view(torch.int16).cpu().numpy().view(np.uint16)
    gv = g.cpu().numpy().reshape(M)
    ref = mo.linear_quantized(abits, *down, group, row_scale=gv, addend=rb)
    e = error_bound(abits, *down, group, False, gv, rb)
    assert np.all(np.abs(h.host_bf16_to_f64(y) - ref) <= e + (np.abs(ref) + e) * 2.0 ** -8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        graph.replay()
        eager = step()[0]
        torch.cuda.synchronize()
        assert torch.equal(got[0], y) and torch.equal(eager, y)


def test_stack_with_routing_rules():
    import torch
    from mixture_experts_ffn_renorm_amd.stack import MoEStack
    moe = _moe()
    M = 24
    shape = wl.WORKLOADS["qwen15"]
    layers = [wl.make_device_layer(shape, M, 1 + i, "cuda", I=128) for i in range(3)]
    for i, lay in enumerate(layers[:2]):
        lay["routing"] = moe.Routing(4, score="sigmoid", n_group=4, topk_group=2, group_top=2,
                                     select_bias=torch.full((60,), 0.01 * i, device="cuda"))
    x = torch.randn((M, 2048), device="cuda").to(torch.bfloat16)
    stack = MoEStack(layers, 4, M)
    y = stack.step(x).clone()
    want = x.clone()
    for lay in layers:
        if lay.get("routing") is not None:
            o, _ = moe.moe_forward_scored(want, lay["w_router"], lay["w13"], lay["w2"],
                                          lay["routing"], logit_bias=lay["logit_bias"])
        else:
            o, _ = moe.moe_forward(want, lay["w_router"], lay["w13"], lay["w2"], 4,
                                   logit_bias=lay["logit_bias"])
        want.add_(o)
    graph, out = stack.capture(x)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert torch.equal(y, want)
    with pytest.raises(ValueError):
        MoEStack([dict(layers[0], routing=moe.Routing(5))], 4, M)
