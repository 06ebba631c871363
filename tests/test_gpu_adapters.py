"""Low-rank adapters on the GPU (moe_linear_adapters) against the float64
oracle, alone and beside the 4-bit projection."""

from __future__ import annotations

import numpy as np
import pytest

import moe_workloads as wl
from oracle import dense_oracle as do
from oracle import moe_oracle as mo
from tests import helpers as h
from tests import test_gpu_qlinear as ql

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
B = 2.0 ** -8      # half a bf16 step, relative


def _moe():
    import mixture_experts_ffn_renorm_amd as moe
    return moe


def bits(a):
    return wl.f32_to_bf16_bits(np.asarray(a, dtype=np.float32))


def wide(b):
    return mo.widen_bf16(b).astype(np.float64)


def inputs(M, S, R, K, N, seed):
    rng = np.random.default_rng(seed)
    return dict(x=bits(rng.standard_normal((M, K))),
                a=bits(rng.standard_normal((S, R, K)) / np.sqrt(K)),
                b=bits(rng.standard_normal((S, N, R)) / np.sqrt(R)),
                scales=(0.5 + rng.random(S)).astype(np.float32),
                addend=bits(rng.standard_normal((M, N))),
                random=rng.integers(-1, S, M).astype(np.int32),
                runs=np.sort(rng.integers(-1, S, M)).astype(np.int32)[::-1].copy())


def reference(d, slots, scaled, added, gated):
    """The result in float64 and its bound: x A^T in fp32 (K / 32 + 64
    roundings in a row), times the scale, kept to 2^-16 of itself (two bf16
    numbers; where it stays fp32 that holds too), t B^T with R terms twice, the
    addend; SiLU as in the products' own tests; one bf16 rounding."""
    x, a, b = wide(d["x"]), wide(d["a"]), wide(d["b"])
    S, K, R = a.shape[0], x.shape[1], a.shape[1]
    sc = d["scales"].astype(np.float64) if scaled else np.ones(S)
    M, N = x.shape[0], b.shape[1]
    y, e = np.zeros((M, N)), np.zeros((M, N))
    for s in set(slots.tolist()):
        if not 0 <= s < S:
            continue
        at = slots == s
        t = x[at] @ a[s].T * sc[s]
        T = np.abs(x[at]) @ np.abs(a[s]).T * abs(sc[s])
        et = T * (K / 32 + 66) * U + np.abs(t) * 2.0 ** -16
        y[at] = t @ b[s].T
        e[at] = et @ np.abs(b[s]).T + (2 * R + 16) * U * ((np.abs(t) + et) @ np.abs(b[s]).T)
    if added:
        ad = wide(d["addend"])
        e = e + U * (np.abs(y) + np.abs(ad) + e)
        y = y + ad
    if gated:
        n = N // 2
        g, u, eg, eu = y[:, :n], y[:, n:], e[:, :n], e[:, n:]
        act = np.abs(g / (1 + np.exp(-g)))
        e = 1.1 * eg * np.abs(u) + act * eu + 1.1 * eg * eu + \
            act * np.abs(u) * (np.abs(g) + 8) * 2 * U
        y = g / (1 + np.exp(-g)) * u
    return y, e + (np.abs(y) + e) * B + 2.0 ** -133


def check(M, S, R, K, N, order="random", seed=0, scaled=True, added=True, gated=False,
          in_place=False, slots=None, data=None):
    import torch
    moe = _moe()
    d = inputs(M, S, R, K, N, seed) if data is None else data
    slots = d[order] if slots is None else slots
    n_out = N // 2 if gated else N
    buf = torch.full((M * n_out + 64,), -7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:M * n_out].view(M, n_out)
    addend = h.dev_bf16(d["addend"]) if added else None
    if in_place:
        out.copy_(addend)
        addend = out
    ad = dict(a=h.dev_bf16(d["a"]), b=h.dev_bf16(d["b"]),
              scales=h.dev_f32(d["scales"]) if scaled else None)
    need = moe.moe_linear_adapters_workspace_size(M, K, R)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")     # NaN everywhere
    got = moe.moe_linear_adapters(h.dev_bf16(d["x"]), ad, h.dev_i32(slots), gated=gated,
                                  addend=addend, out=out, ws=ws[:need])
    torch.cuda.synchronize()
    assert got is out and (buf[M * n_out:] == -7.0).all() and (ws[need:] == 255).all()
    ref, bound = reference(d, slots, scaled, added, gated)
    plain = do.adapters(wide(d["x"]), wide(d["a"]), wide(d["b"]), d["scales"] if scaled else None,
                        slots, wide(d["addend"]) if added else None, gated)
    err = np.abs(h.host_bf16_to_f64(out) - plain)
    assert np.abs(ref - plain).max() <= 1e-9 * (1 + np.abs(plain).max())
    assert np.all(err <= bound), (err / bound).max()
    return out


MS = [1, 2, 5, 16, 17, 31, 64, 65, 66, 100, 128, 129, 130, 300, 1000, 1030]


@pytest.mark.parametrize("order", ["random", "runs"])
@pytest.mark.parametrize("M", MS)
def test_batches(M, order):
    check(M, 5, 16, 128, 136, order, seed=M)


@pytest.mark.parametrize("M", [1, 40, 200])
@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 48, 64, 72, 96, 120, 128])
def test_ranks(R, M):
    check(M, 4, R, 96, 72, seed=R)
    check(M, 4, R, 96, 96, seed=R, gated=True)


@pytest.mark.parametrize("M", [1, 30, 130, 135])
@pytest.mark.parametrize("K", [8, 16, 24, 32, 40, 64, 248, 256, 264, 504, 520, 1408, 2048, 8192])
def test_inner_sizes(K, M):
    check(M, 3, 16, K, 40, seed=K)


@pytest.mark.parametrize("M", [1, 30, 130, 135])
@pytest.mark.parametrize("N", [8, 16, 24, 56, 64, 72, 248, 256, 264, 520, 2048, 11264])
def test_output_sizes(N, M):
    check(M, 3, 16, 64, N, seed=N)
    if N % 16 == 0:
        check(M, 3, 16, 64, N, seed=N, gated=True)


@pytest.mark.parametrize("M", [3, 64, 65, 260, 1100])
@pytest.mark.parametrize("scaled,added,gated,in_place", [
    (False, True, False, False), (True, False, False, False), (True, True, False, True),
    (False, False, False, False), (True, True, True, False), (True, False, True, False)])
def test_epilogues(M, scaled, added, gated, in_place):
    check(M, 6, 24, 72, 80, "random", 3, scaled, added, gated, in_place)
    check(M, 6, 24, 72, 80, "runs", 4, scaled, added, gated, in_place)


@pytest.mark.parametrize("M", [2, 64, 70, 140, 500])
def test_slots(M):
    """No adapter at all, all one, each its own, numbers far outside."""
    S = 500
    d = inputs(M, S, 8, 40, 48, 7)
    rng = np.random.default_rng(2)
    far = rng.choice([-2 ** 31, -5, -1, S, S + 1, 2 ** 31 - 1, 0, S - 1], M)
    for slots in (np.full(M, -1), np.full(M, S - 1), rng.permutation(S)[:M], far):
        for kw in (dict(), dict(in_place=True), dict(gated=True), dict(added=False)):
            check(M, S, 8, 40, 48, data=d, slots=slots.astype(np.int32), **kw)


@pytest.mark.parametrize("S", [1, 63, 64, 1024, 4096])
def test_many_adapters(S):
    check(150, S, 8, 32, 40, seed=S)
    check(9000, min(S, 70), 8, 16, 16, seed=S)           # two windows of the grouping


@pytest.mark.parametrize("order", ["random", "runs"])
def test_many_rows(order):
    check(20000, 30, 16, 24, 24, order, seed=2)


@pytest.mark.parametrize("M", [1, 7])
@pytest.mark.parametrize("R,K,N", [(16, 2048, 2048), (16, 2056, 2048), (128, 256, 528), (128, 264, 528),
                                   (40, 800, 272), (8, 4096, 4112)])
def test_one_and_two_launches(R, K, N, M):
    """At the border of the one-launch form, and just past it."""
    for gated in (False, True):
        check(M, 3, R, K, N, seed=R, gated=gated)


@pytest.mark.parametrize("M,order", [(64, "random"), (1000, "runs"), (700, "random")])
def test_layer_sizes(M, order):
    check(M, 8, 64, 2048, 2048, order, seed=1)


@pytest.mark.parametrize("M", [3, 180])
def test_a_row_that_is_not_finite_stays_alone(M):
    import torch
    moe = _moe()
    d = inputs(M, 2, 16, 64, 32, 5)
    ad = dict(a=h.dev_bf16(d["a"]), b=h.dev_bf16(d["b"]))
    x, slots, add = h.dev_bf16(d["x"]), h.dev_i32(np.zeros(M)), h.dev_bf16(d["addend"])
    good = moe.moe_linear_adapters(x, ad, slots, addend=add)
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[1, 63] = bad
        out = moe.moe_linear_adapters(y, ad, slots, addend=add)
        torch.cuda.synchronize()
        assert not torch.isfinite(out[1]).any()
        assert torch.equal(out[2:], good[2:]) and torch.equal(out[0], good[0])
    # an adapter that is not finite reaches its own rows alone
    ad["a"][1, 0, 0] = float("nan")
    ad["b"][1, 0, 0] = float("nan")
    out = moe.moe_linear_adapters(x, ad, slots, addend=add)
    assert torch.equal(out, good)


def test_beside_the_quantized_projection():
    """A shared expert with adapters: 4-bit gate and up rows, their adapters and
    the activation, 4-bit down rows, their adapters added in place."""
    import torch
    moe = _moe()
    for M in (1, 48, 300):
        H, I, S, R, group = 256, 128, 5, 16, 64
        up, down = inputs(M, S, R, H, 2 * I, M), inputs(M, S, R, I, H, M + 1)
        x, slots = h.dev_bf16(up["x"]), h.dev_i32(up["random"])
        w13, w2 = ql.matrix(2 * I, H, group, 1), ql.matrix(H, I, group, 2)
        ad13, ad2 = (dict(a=h.dev_bf16(d["a"]), b=h.dev_bf16(d["b"]), scales=h.dev_f32(d["scales"]))
                     for d in (up, down))
        y = moe.moe_linear_quantized(x, ql.to_device(*w13, group))
        act = moe.moe_linear_adapters(x, ad13, slots, gated=True, addend=y)
        out = moe.moe_linear_quantized(act, ql.to_device(*w2, group))
        out = moe.moe_linear_adapters(act, ad2, slots, addend=out, out=out)
        torch.cuda.synchronize()
        # each step from the bits that the one before left
        ref_y = mo.linear_quantized(up["x"], *w13, group)
        got_y = h.host_bf16_to_f64(y)
        assert np.abs(got_y - ref_y).max() <= 0.02 * np.abs(ref_y).max()
        d = dict(up, addend=y.view(torch.int16).cpu().numpy().view(np.uint16))
        ref, bound = reference(d, up["random"], True, True, True)
        assert np.all(np.abs(h.host_bf16_to_f64(act) - ref) <= bound)
        a_bits = act.view(torch.int16).cpu().numpy().view(np.uint16)
        shared = mo.linear_quantized(a_bits, *w2, group)
        d = dict(down, x=a_bits, addend=bits(shared))
        ref, bound = reference(d, up["random"], True, True, False)
        # the projection's own rounding to bf16 once more (its fp32 sums differ
        # from float64 by far less than a bf16 step, but may round to a neighbour)
        assert np.all(np.abs(h.host_bf16_to_f64(out) - ref) <= bound + np.abs(shared) * 2 * B + 1e-5)


@pytest.mark.parametrize("M", [1, 48, 300])
def test_repeatable_captured_and_on_two_streams(M):
    import torch
    moe = _moe()
    data = []
    for i in range(2):
        d = inputs(M, 7, 32, 264, 520, 20 + i)
        data.append((h.dev_bf16(d["x"]), dict(a=h.dev_bf16(d["a"]), b=h.dev_bf16(d["b"])),
                     h.dev_i32(d["random"]), h.dev_bf16(d["addend"])))

    def call(t, stream=None):
        return moe.moe_linear_adapters(t[0], t[1], t[2], addend=t[3], stream=stream)

    want = [call(t) for t in data]
    torch.cuda.synchronize()
    graphs = []
    for t in data:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(t)
        graphs.append((g, out))
    for _ in range(3):
        for (g, out), exp in zip(graphs, want):
            out.zero_()
            g.replay()
            again = call(data[0])
            torch.cuda.synchronize()
            assert torch.equal(out, exp) and torch.equal(again, want[0])
    streams = [torch.cuda.Stream() for _ in data]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    out = [[call(t, s) for t, s in zip(data, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for rnd in out for a, b in zip(rnd, want))


def test_a_workspace_serves_fewer_rows():
    moe = _moe()
    for K, R in ((64, 8), (2048, 128)):
        sizes = [moe.moe_linear_adapters_workspace_size(M, K, R) for M in
                 (0, 1, 5, 64, 65, 129, 500, 4096, 8192, 8193, 20000, 2 ** 21 - 1)]
        assert sizes == sorted(sizes) and sizes[0] > 0


def test_binding_refuses_wrong_tensors():
    import torch
    moe = _moe()
    d = inputs(6, 3, 16, 64, 48, 2)
    x, slots, add = h.dev_bf16(d["x"]), h.dev_i32(d["random"]), h.dev_bf16(d["addend"])
    ad = dict(a=h.dev_bf16(d["a"]), b=h.dev_bf16(d["b"]), scales=h.dev_f32(d["scales"]))
    good = moe.moe_linear_adapters(x, ad, slots)
    assert good.shape == (6, 48)
    for bad in (x.float(), x[:, ::2], x[:, :32].contiguous(), x.t().contiguous().t()):
        with pytest.raises((ValueError, moe.MoeError)):
            moe.moe_linear_adapters(bad, ad, slots)
    for change in (dict(a=ad["a"][:2]), dict(b=ad["b"][:, :, :8].contiguous()),
                   dict(scales=ad["scales"][:2]), dict(scales=ad["scales"].double()),
                   dict(a=ad["a"][:, :12].contiguous(), b=ad["b"][:, :, :12].contiguous())):
        with pytest.raises((ValueError, moe.MoeError)):
            moe.moe_linear_adapters(x, dict(ad, **change), slots)
    for bad in (slots.long(), slots[:5], slots.cpu()):
        with pytest.raises(ValueError):
            moe.moe_linear_adapters(x, ad, bad)
    with pytest.raises(ValueError):
        moe.moe_linear_adapters(x, ad, slots, addend=add[:, :40].contiguous())
    with pytest.raises(moe.MoeError):
        moe.moe_linear_adapters(x, ad, slots, ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.moe_linear_adapters(x, ad, slots, addend=add, gated=True,
                                out=add.view(-1)[:6 * 24].view(6, 24))
    assert moe.moe_linear_adapters(x[:0], ad, slots[:0]).shape == (0, 48)
