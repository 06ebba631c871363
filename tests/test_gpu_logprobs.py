"""Token log probabilities on the GPU (moe_token_logprobs and its gradient)
against the float64 oracle."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import dense_oracle as do

pytestmark = pytest.mark.gpu

U = 2.0 ** -24     # half an fp32 step


def _moe():
    import mixture_experts_ffn_renorm_amd as moe
    return moe


def draw(M, V, seed, std=2.5):
    return (np.random.default_rng(seed).standard_normal((M, V)) * std).astype(np.float32)


def device(l, dtype):
    """The logits on the device in a type, and as that type holds them."""
    import torch
    d = torch.from_numpy(np.ascontiguousarray(l)).to(getattr(torch, dtype)).cuda()
    return d, d.float().cpu().numpy()


def bounds(l):
    """Largest fp32 errors of lse, entropy and (l - lse) per row.

    With x = l - m <= 0: e^x is formed from fp32((l - m) log2 e), off by at
    most 3 U |x| in x (difference, product, constant), by 2^-23 in the
    exponential; the sums run over at most 64 terms in a register, 6 + 8 + 64
    + 6 joins of lanes, waves and chunks and one factor: 160 roundings cover
    them.  So z is off by (3 A + 162) U relatively, A = sum p |x|, and with
    one more product per term s = sum p x by sum p |x| (6 |x| + 165) U.
    """
    l = np.where(np.isnan(l).any(axis=1, keepdims=True), 0.0, l.astype(np.float64))   # NaN rows: any
    m = l.max(axis=1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    x = np.clip(l - m, -800.0, 0.0)
    p = np.exp(x)
    z = p.sum(axis=1)
    z = np.where(z > 0, z, 1.0)
    p = p / z[:, None]
    A, B = (p * -x).sum(axis=1), (p * x * x).sum(axis=1)
    dz = (3 * A + 162) * U
    lz = np.log(z)
    ds = (6 * B + 165 * A) * U + A * dz
    lse = dz + U * (2 * np.abs(lz) + np.abs(m[:, 0] + lz))
    ent = dz + ds + U * (4 * np.abs(lz) + 4 * A + 2 * np.abs(lz + A))
    return lse + 1e-37, ent + 1e-37, dz + U * 2 * np.abs(lz) + 1e-37


def check(l, dtype, top, tokens=None, seed=0):
    import torch
    moe = _moe()
    d, l = device(l, dtype)
    M, V = l.shape
    if tokens is None:
        tokens = np.random.default_rng(seed + 1).integers(0, V, M)
    tok = torch.from_numpy(tokens.astype(np.int32)).cuda()
    got = moe.moe_token_logprobs(d, tok, top=top)
    torch.cuda.synchronize()
    ref = do.token_logprobs(l, tokens, top)
    el, ee, ep = bounds(l)
    with np.errstate(invalid="ignore"):
        for name, t, e in (("logprobs", got[0], ep + 3 * U * np.abs(ref["logprobs"])),
                           ("entropy", got[1], ee), ("lse", got[2], el)):
            compare(name, t.cpu().numpy(), ref[name], e)
        if top:
            assert np.array_equal(got[3].cpu().numpy(), ref["top_ids"])
            compare("top_logprobs", got[4].cpu().numpy(), ref["top_logprobs"],
                    ep[:, None] + 3 * U * np.abs(ref["top_logprobs"]))
        else:
            assert got[3] is None and got[4] is None
    return got


def compare(name, got, ref, e):
    got = got.astype(np.float64)
    assert got.shape == ref.shape
    # outputs are fp32: what lies past its largest number rounds to infinity
    # (-3e38 - 3e38 has no other fp32 value than -inf)
    with np.errstate(over="ignore"):
        same = (got == ref) | (got == ref.astype(np.float32)) | (np.isnan(got) & np.isnan(ref))
    bad = ~same & ~(np.abs(got - ref) <= e)
    assert not bad.any(), (name, np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3])


DTYPES = ["bfloat16", "float32"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 2, 3, 5, 7, 8, 9, 31, 64, 65, 1000, 4095, 4097, 32003, 50257,
                               131072, 151937])
@pytest.mark.parametrize("M", [1, 5])
def test_sizes(V, M, dtype):
    check(draw(M, V, V + M), dtype, min(V, 7), seed=V)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,V", [(300, 4099), (700, 1003), (130, 40001), (2100, 257)])
def test_many_rows(M, V, dtype):
    check(draw(M, V, 3), dtype, 5)
    check(draw(M, V, 4, 0.0), dtype, 3)      # all equal


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("top", [0, 1, 2, 5, 20, 31, 32])
@pytest.mark.parametrize("M,V", [(1, 131072), (3, 33), (33, 20011)])
def test_alternatives(M, V, top, dtype):
    check(draw(M, V, top), dtype, top)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [40, 5000, 131072])
def test_ties_go_to_the_lower_id(V, dtype):
    rng = np.random.default_rng(V)
    l = np.round(draw(4, V, 5)) * 1.0                    # few different values
    check(l, dtype, 32)
    l = np.zeros((3, V), np.float32)                     # one value, then two, then signed zeros
    l[1, rng.integers(0, V, 5)] = 1.0
    l[2, ::2] = -0.0
    check(l, dtype, 32)
    l = -np.ones((2, V), np.float32) * 7.25              # ties of negative numbers
    l[1, ::3] = -7.0
    check(l, dtype, 32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [300, 20011, 131072])
def test_rows_in_order(V, dtype):
    """Every logit passes the threshold of those before it, or none does."""
    up = np.linspace(-6, 6, V, dtype=np.float32)
    check(np.stack([up, up[::-1], -np.abs(up), np.abs(up)]), dtype, 20)


LOWEST = {"bfloat16": -3.3895313892515355e38, "float32": np.finfo(np.float32).min}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("low", ["inf", "lowest", -1e9, -1e4])
@pytest.mark.parametrize("V", [37, 8193, 70001])
def test_masks(V, low, dtype):
    """Tokens ruled out by -inf, the type's lowest value or a large negative
    number: many, all but one, all; the token asked for among them."""
    v = -np.inf if low == "inf" else LOWEST[dtype] if low == "lowest" else low
    l = draw(6, V, 9)
    rng = np.random.default_rng(1)
    l[0, rng.random(V) < 0.5] = v
    l[1, :] = v
    l[1, V // 2] = 1.5
    l[2, :] = v
    l[3, :V // 2] = v
    l[4, V // 2:] = v
    tokens = np.array([int(np.argmin(l[0])), 0, 3, V - 1, V - 1, V // 3])
    check(l, dtype, 32, tokens)


@pytest.mark.parametrize("dtype", DTYPES)
def test_far_logits(dtype):
    """Offsets far from 0, a peaked row, logits whose difference overflows."""
    l = draw(5, 3001, 2)
    l[0] += 20000
    l[1] -= 1e30
    l[2, 77] = 90.0
    l[3] *= 40
    l[4, :3] = [3e38, -3e38, 2.9e38]
    check(l, dtype, 9, np.array([5, 6, 77, 8, 1]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [12, 9001])
def test_rows_that_are_not_finite(V, dtype):
    l = draw(7, V, 6)
    l[1, 3] = np.nan
    l[2, 5] = np.inf
    l[3, :] = np.nan
    l[4, :] = -np.inf
    l[4, 2] = np.nan
    l[5, 1:4] = [np.inf, np.nan, -np.inf]
    check(l, dtype, 9)


@pytest.mark.parametrize("dtype", DTYPES)
def test_tokens_outside(dtype):
    got = check(draw(5, 100, 7), dtype, 2, np.array([-1, 100, 2 ** 31 - 1, -2 ** 31, 99]))
    assert got[0][:4].eq(0).all() and got[0][4] != 0


def test_rows_past_32_bits():
    """Rows whose first logit is more than 2^31 elements into the tensor."""
    import torch
    moe = _moe()
    M, V = 70000, 32771
    l = torch.zeros((M, V), dtype=torch.bfloat16, device="cuda")
    pick = [0, 1, 40000, 65535, 65537, M - 1]
    rows = draw(len(pick), V, 8)
    d, rows = device(rows, "bfloat16")
    l[pick] = d
    tokens = torch.arange(M, dtype=torch.int32, device="cuda") % V
    lp, ent, lse, ids, tlp = moe.moe_token_logprobs(l, tokens, top=3)
    ref = do.token_logprobs(rows, np.array([p % V for p in pick]), 3)
    el, ee, ep = bounds(rows)
    compare("logprobs", lp[pick].cpu().numpy(), ref["logprobs"], ep + 3 * U * np.abs(ref["logprobs"]))
    compare("entropy", ent[pick].cpu().numpy(), ref["entropy"], ee)
    assert np.array_equal(ids[pick].cpu().numpy(), ref["top_ids"])
    g = torch.zeros(M, device="cuda")
    g[pick] = 1.0
    grad = moe.moe_token_logprobs_backward(l, tokens, lse, ent, g, g, grad_logits=l)
    assert grad is l
    want = do.token_logprobs_backward(rows, np.array([p % V for p in pick]), lse[pick].cpu().numpy(),
                                      ent[pick].cpu().numpy(), np.ones(len(pick)), np.ones(len(pick)))
    got = grad[pick].double().cpu().numpy()
    compare("grad", got, want, grad_bound(rows, lse[pick].cpu().numpy(), ent[pick].cpu().numpy(),
                                          np.ones(len(pick)), np.ones(len(pick)), want, "bfloat16"))
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[pick] = False
    for r in torch.split(rest.nonzero()[:, 0], 8192):
        assert not grad[r].any()


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------

def grad_bound(l, lse, ent, g, h, ref, dtype):
    """log p = fp32(l - lse) is off by U |log p|, its exponent by 2 U more of
    that, the exponential by 2^-23: p by (3 |log p| + 3) U; the inner sum by
    three roundings of its terms; two more products, a sum at the token; the
    type's rounding."""
    with np.errstate(invalid="ignore", over="ignore"):
        logp = np.maximum(l.astype(np.float64) - lse[:, None], -800.0)
        p = np.exp(np.minimum(logp, 0.1))
        terms = np.abs(g)[:, None] + np.abs(h)[:, None] * (np.abs(logp) + np.abs(ent)[:, None])
        e = p * terms * (3 * np.abs(logp) + 10) * U + U * np.abs(g)[:, None] * 2
        half = 2.0 ** -8 if dtype == "bfloat16" else U
        return np.nan_to_num(e, nan=0.0) * (1 + half) + half * np.abs(ref) + 1e-37


def check_grad(l, dtype, tokens=None, entropy=True, seed=0, in_place=False):
    import torch
    moe = _moe()
    d, l = device(l, dtype)
    M, V = l.shape
    rng = np.random.default_rng(seed)
    if tokens is None:
        tokens = rng.integers(0, V, M)
    tok = torch.from_numpy(tokens.astype(np.int32)).cuda()
    g, h = rng.standard_normal((2, M)).astype(np.float32)
    lp, ent, lse, _, _ = moe.moe_token_logprobs(d, tok)
    gd, hd = torch.from_numpy(g).cuda(), torch.from_numpy(h).cuda() if entropy else None
    kw = {}
    if in_place:
        kw["grad_logits"] = d
    else:
        guard = torch.full((M * V + 64,), -7.0, dtype=d.dtype, device="cuda")
        kw["grad_logits"] = guard[:M * V].view(M, V)
    out = moe.moe_token_logprobs_backward(d, tok, lse, ent if entropy else None, gd, hd, **kw)
    torch.cuda.synchronize()
    if not in_place:
        assert (guard[M * V:] == -7.0).all()
    if not entropy:
        h = np.zeros(M, np.float32)
    lse, ent = lse.cpu().numpy(), ent.cpu().numpy()
    with np.errstate(invalid="ignore", over="ignore"):
        ref = do.token_logprobs_backward(l, tokens, lse, ent, g, h)
    got = out.double().cpu().numpy()
    compare("grad", got, ref, grad_bound(l, lse, ent, g, h, ref, dtype))
    return got, l, g, h


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("entropy", [True, False])
@pytest.mark.parametrize("M,V", [(1, 1), (1, 7), (3, 9), (5, 1000), (61, 32003), (2, 131072),
                                 (900, 517), (7, 50257)])
def test_gradient(M, V, entropy, dtype):
    check_grad(draw(M, V, 11), dtype, entropy=entropy)
    check_grad(draw(M, V, 12), dtype, entropy=entropy, in_place=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("low", ["inf", "lowest"])
def test_gradient_under_masks(low, dtype):
    v = -np.inf if low == "inf" else LOWEST[dtype]
    V = 2003
    l = draw(6, V, 13)
    l[0, ::2] = v
    l[1, :] = v
    l[2, :] = v
    l[2, 9] = 0.25
    tokens = np.array([0, 4, 9, -1, V, 5])      # a masked one, a masked row's, the only one, outside
    got, _, _, _ = check_grad(l, dtype, tokens)
    assert not got[1].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("low", ["inf", "lowest"])
def test_gradient_of_a_masked_row_is_zero_for_any_that_comes_in(low, dtype):
    import torch
    moe = _moe()
    l = draw(3, 1003, 17)
    l[1, :] = -np.inf if low == "inf" else LOWEST[dtype]
    d, l = device(l, dtype)
    tok = torch.tensor([3, 4, 5], dtype=torch.int32, device="cuda")
    _, ent, lse, _, _ = moe.moe_token_logprobs(d, tok)
    g = torch.ones(3, device="cuda")
    want = moe.moe_token_logprobs_backward(d, tok, lse, ent, g, g)
    for bad in (np.nan, np.inf):
        b = torch.tensor([1.0, bad, 1.0], device="cuda")
        got = moe.moe_token_logprobs_backward(d, tok, lse, ent, b, b)
        assert not got[1].any() and torch.equal(got, want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_of_rows_that_are_not_finite_stays_alone(dtype):
    l = draw(4, 333, 14)
    l[1, 7] = np.nan
    l[2, 9] = np.inf
    got, _, _, _ = check_grad(l, dtype)
    assert np.isnan(got[1:3]).all() and np.isfinite(got[[0, 3]]).all()


def test_gradient_against_differences():
    """Central differences of the forward pass's own definition."""
    l = draw(3, 50, 15, 1.0)
    tokens = np.array([3, 20, 49])
    got, l, g, h = check_grad(l, "float32", tokens)
    eps = 1e-5
    l = l.astype(np.float64)

    def value(l):
        r = do.token_logprobs(l, tokens)
        return r["logprobs"] * g + r["entropy"] * h

    for v in range(50):
        step = np.zeros_like(l)
        step[:, v] = eps
        d = (value(l + step) - value(l - step)) / (2 * eps)
        # differences: eps^2 of the third derivative (below 20 here) and
        # 2^-52 * 20 / eps of cancellation; the kernel's own error as above
        assert np.abs(d - got[:, v]).max() < 2e-9 + 1e-9 + 100 * U


# ---------------------------------------------------------------------------
# streams, graphs, refusals
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M,V", [(1, 131072), (300, 4099)])
def test_repeatable_captured_and_on_two_streams(M, V):
    import torch
    moe = _moe()
    d = [device(draw(M, V, 20 + i), "bfloat16")[0] for i in range(2)]
    tok = torch.arange(M, dtype=torch.int32, device="cuda")
    g = torch.ones(M, device="cuda")

    def both(l, stream=None):
        f = moe.moe_token_logprobs(l, tok, top=4, stream=stream)
        b = moe.moe_token_logprobs_backward(l, tok, f[2], f[1], g, g, stream=stream)
        return (*f, b)

    want = [both(l) for l in d]
    torch.cuda.synchronize()
    graphs = []
    for l in d:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = both(l)
        graphs.append((gr, out))
    for _ in range(3):
        for (gr, out), exp in zip(graphs, want):
            for t in out:
                t.zero_()
            gr.replay()
            again = both(d[0])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, exp))
            assert all(torch.equal(a, b) for a, b in zip(again, want[0]))
    streams = [torch.cuda.Stream() for _ in d]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    out = [[both(l, stream=s) for l, s in zip(d, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for rnd in out:
        for a, b in zip(rnd, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_binding_refuses_wrong_tensors():
    import torch
    moe = _moe()
    l = torch.zeros((4, 64), device="cuda")
    tok = torch.zeros(4, dtype=torch.int32, device="cuda")
    f = torch.zeros(4, device="cuda")
    for bad in (l.half(), l.double(), l[:, ::2], l.t().contiguous().t(), l[:, :0]):
        with pytest.raises((ValueError, moe.MoeError)):
            moe.moe_token_logprobs(bad, tok)
        with pytest.raises((ValueError, moe.MoeError)):
            moe.moe_token_logprobs_backward(bad, tok, f, f, f, f)
    for bad in (tok.long(), tok[:3], tok.cpu()):
        with pytest.raises(ValueError):
            moe.moe_token_logprobs(l, bad)
        with pytest.raises(ValueError):
            moe.moe_token_logprobs_backward(l, bad, f, f, f, f)
    for top in (-1, 33, 65):
        with pytest.raises(moe.MoeError):
            moe.moe_token_logprobs(l, tok, top=top)
    with pytest.raises(moe.MoeError):
        moe.moe_token_logprobs(l, tok, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.moe_token_logprobs(l, tok, logprobs=f, entropy=f)
    with pytest.raises(ValueError):
        moe.moe_token_logprobs_backward(l, tok, f, None, f, f)
    with pytest.raises(ValueError):
        moe.moe_token_logprobs_backward(l, tok, f, f, f, f, grad_logits=l.bfloat16())
    assert moe.moe_token_logprobs(l[:0], tok[:0], top=2)[3].shape == (0, 2)
    assert moe.moe_token_logprobs_backward(l[:0], tok[:0], f[:0], f[:0], f[:0]).shape == (0, 64)
