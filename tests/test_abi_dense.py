"""Argument checks of the gated block, the adapters and the token log
probabilities on the CPU: every call here is rejected, or has nothing to do,
before any launch."""

from __future__ import annotations

import ctypes

import pytest

NULL = None
A = 0x100000000          # never dereferenced
STEP = 0x100000          # more than any operand here
BIG = 1 << 40


def _moe():
    import mixture_experts_ffn_renorm_amd as moe
    return moe


def at(i):
    return A + i * STEP


# ---------------------------------------------------------------------------
# gated block
# ---------------------------------------------------------------------------

GATED = dict(x=at(0), w=at(1), M=4, H=64, I=24, out=at(2))


def gated(**change):
    a = dict(GATED, **change)
    return _moe().library().moe_linear_gated(a["x"], a["w"], a["M"], a["H"], a["I"], a["out"], NULL)


def test_gated_refusals():
    for change, status in (
            (dict(M=-1), -1), (dict(H=0), -1), (dict(I=0), -1), (dict(H=60), -2), (dict(I=12), -2),
            (dict(M=1 << 21), -2), (dict(H=(1 << 17) + 8), -2), (dict(I=(1 << 17) + 8), -2),
            (dict(M=0, x=NULL, w=NULL, out=NULL), 0),
            (dict(x=NULL), -1), (dict(w=NULL), -1), (dict(out=NULL), -1),
            (dict(x=at(0) + 8), -1), (dict(w=at(1) + 2), -1), (dict(out=at(2) + 4), -1),
            (dict(out=at(0)), -1), (dict(out=at(1) + 2 * 24 * 64 * 2 - 16), -1),
            (dict(out=at(1) - 4 * 24 * 2 + 16), -1)):
        assert gated(**change) == status, change


def backward(**change):
    a = dict(GATED, d=at(3), gx=at(4), gw=at(5), ws=at(16), n=BIG)
    a.update(change)
    return _moe().library().moe_linear_gated_backward(
        a["x"], a["w"], a["d"], a["M"], a["H"], a["I"], a["gx"], a["gw"], a["ws"], a["n"], NULL)


def test_gated_backward_refusals():
    need = _moe().moe_linear_gated_backward_workspace_size(4, 64, 24)
    assert need >= 4 * 48 * 2
    for change, status in (
            (dict(M=-1), -1), (dict(H=60), -2), (dict(I=12), -2), (dict(M=1 << 21), -2),
            (dict(x=NULL), -1), (dict(w=NULL), -1), (dict(d=NULL), -1), (dict(gx=NULL, gw=NULL), -1),
            (dict(x=at(0) + 8), -1), (dict(d=at(3) + 2), -1), (dict(gx=at(4) + 2), -1),
            (dict(gw=at(5) + 8), -1), (dict(ws=at(16) + 8), -1),
            (dict(ws=NULL), -3), (dict(n=need - 1), -3),
            (dict(gx=at(0)), -1), (dict(gx=at(3)), -1), (dict(gw=at(1)), -1), (dict(gw=at(4)), -1),
            (dict(ws=at(4)), -1), (dict(ws=at(0)), -1), (dict(gx=at(16) + 64), -1),
            (dict(M=0, gx=NULL, gw=NULL, x=NULL, w=NULL, d=NULL, ws=NULL), 0),
            (dict(M=0, gw=NULL, x=NULL, w=NULL, d=NULL, ws=NULL), 0)):
        assert backward(**change) == status, change


def test_gated_workspace_sizes():
    size = _moe().moe_linear_gated_backward_workspace_size
    for bad in ((-1, 64, 24), (4, 60, 24), (4, 64, 20), (4, 0, 24), (1 << 21, 64, 24), (1 << 33, 64, 24)):
        assert size(*bad) == 0
    assert size(0, 64, 24) > 0


# ---------------------------------------------------------------------------
# adapters
# ---------------------------------------------------------------------------

ADAPTERS = dict(x=at(0), a=at(1), b=at(2), scales=at(3), slots=at(4), count=5, rank=16, M=4, K=64,
                N=48, gated=0, addend=at(6), out=at(7), ws=at(16), n=BIG)


def adapters(**change):
    moe = _moe()
    v = dict(ADAPTERS, **change)
    w = moe.Adapters(v["count"], v["rank"], v["a"], v["b"], v["scales"])
    return moe.library().moe_linear_adapters(
        v["x"], ctypes.addressof(w), v["slots"], v["M"], v["K"], v["N"], v["gated"], v["addend"],
        v["out"], v["ws"], v["n"], NULL)


def test_adapters_refusals():
    need = _moe().moe_linear_adapters_workspace_size(4, 64, 16)
    for change, status in (
            (dict(M=-1), -1), (dict(K=0), -1), (dict(N=0), -1), (dict(rank=0), -1), (dict(count=0), -1),
            (dict(gated=2), -1), (dict(K=60), -2), (dict(N=44), -2), (dict(N=56, gated=1), -2),
            (dict(rank=12), -2), (dict(rank=136), -2), (dict(count=4097), -2), (dict(M=1 << 21), -2),
            (dict(K=(1 << 17) + 8), -2), (dict(N=(1 << 17) + 8), -2),
            (dict(M=0, x=NULL, out=NULL, ws=NULL), 0),
            (dict(x=NULL), -1), (dict(a=NULL), -1), (dict(b=NULL), -1), (dict(slots=NULL), -1),
            (dict(out=NULL), -1), (dict(x=at(0) + 8), -1), (dict(a=at(1) + 8), -1),
            (dict(b=at(2) + 8), -1), (dict(addend=at(6) + 8), -1), (dict(out=at(7) + 8), -1),
            (dict(ws=at(16) + 8), -1), (dict(ws=NULL), -3), (dict(n=need - 1), -3),
            (dict(out=at(0)), -1), (dict(out=at(1)), -1), (dict(out=at(2)), -1), (dict(out=at(3)), -1),
            (dict(out=at(4)), -1), (dict(out=at(6) + 16), -1), (dict(out=at(6), gated=1), -1),
            (dict(ws=at(0)), -1), (dict(ws=at(7)), -1), (dict(ws=at(4)), -1)):
        assert adapters(**change) == status, change
    assert _moe().library().moe_linear_adapters(at(0), NULL, at(4), 4, 64, 48, 0, NULL, at(7),
                                                at(16), BIG, NULL) == -1


def test_adapters_workspace_sizes():
    size = _moe().moe_linear_adapters_workspace_size
    for bad in ((-1, 64, 16), (4, 60, 16), (4, 64, 12), (4, 64, 136), (4, 64, 0), (1 << 21, 64, 16),
                (4, 1 << 33, 16)):
        assert size(*bad) == 0
    assert 0 < size(0, 64, 16) <= size(1, 64, 16)


def test_packed_adapters_are_the_struct():
    moe = _moe()
    assert moe._pack_matrix(5, 16, 0x1230, 0x4560, 0x7890) == bytes(
        moe.Adapters(5, 16, 0x1230, 0x4560, 0x7890))


# ---------------------------------------------------------------------------
# token log probabilities
# ---------------------------------------------------------------------------

LOGPROBS = dict(l=at(0), fp32=1, tok=at(1), M=4, V=1000, top=3, lp=at(2), ent=at(3), lse=at(4),
                ids=at(5), tlp=at(6), ws=at(16), n=BIG)


def logprobs(**change):
    v = dict(LOGPROBS, **change)
    return _moe().library().moe_token_logprobs(
        v["l"], v["fp32"], v["tok"], v["M"], v["V"], v["top"], v["lp"], v["ent"], v["lse"], v["ids"],
        v["tlp"], v["ws"], v["n"], NULL)


def test_logprobs_refusals():
    need = _moe().moe_token_logprobs_workspace_size(4, 1000, 3, True)
    for change, status in (
            (dict(M=-1), -1), (dict(V=0), -1), (dict(fp32=2), -1), (dict(top=-1), -1),
            (dict(top=1001), -1), (dict(top=33), -2), (dict(V=2, top=3), -1),
            (dict(V=(1 << 19) + 1), -2), (dict(M=1 << 21), -2), (dict(M=(1 << 20), V=1 << 18), -2),
            (dict(M=0, l=NULL, lp=NULL, ws=NULL), 0),
            (dict(l=NULL), -1), (dict(tok=NULL), -1), (dict(lp=NULL), -1), (dict(ent=NULL), -1),
            (dict(lse=NULL), -1), (dict(ids=NULL), -1), (dict(tlp=NULL), -1),
            (dict(l=at(0) + 4), -1), (dict(ws=at(16) + 8), -1), (dict(ws=NULL), -3),
            (dict(n=need - 1), -3),
            (dict(lp=at(0)), -1), (dict(ent=at(1)), -1), (dict(lse=at(3) + 12), -1),
            (dict(ids=at(6)), -1), (dict(tlp=at(0) + 4 * 4000 - 4), -1), (dict(ws=at(0)), -1),
            (dict(ws=at(2)), -1), (dict(lp=at(16)), -1)):
        assert logprobs(**change) == status, change


def logprobs_backward(**change):
    v = dict(l=at(0), fp32=0, tok=at(1), lse=at(2), ent=at(3), g=at(4), h=at(5), M=4, V=1000,
             out=at(6))
    v.update(change)
    return _moe().library().moe_token_logprobs_backward(
        v["l"], v["fp32"], v["tok"], v["lse"], v["ent"], v["g"], v["h"], v["M"], v["V"], v["out"],
        NULL)


def test_logprobs_backward_refusals():
    for change, status in (
            (dict(M=-1), -1), (dict(V=0), -1), (dict(fp32=-1), -1), (dict(V=(1 << 19) + 1), -2),
            (dict(M=1 << 21), -2), (dict(M=0, l=NULL, out=NULL), 0),
            (dict(l=NULL), -1), (dict(tok=NULL), -1), (dict(lse=NULL), -1), (dict(ent=NULL), -1),
            (dict(g=NULL), -1), (dict(out=NULL), -1), (dict(l=at(0) + 2), -1), (dict(out=at(6) + 8), -1),
            (dict(out=at(0) + 16), -1), (dict(out=at(1)), -1), (dict(out=at(2)), -1),
            (dict(out=at(3)), -1), (dict(out=at(4)), -1), (dict(out=at(5) - 16), -1)):
        assert logprobs_backward(**change) == status, change


def test_logprobs_workspace_sizes():
    size = _moe().moe_token_logprobs_workspace_size
    for bad in ((-1, 1000), (4, 0), (4, 1000, 33), (4, 20, 21), (4, 1000, -1), (1 << 21, 1000),
                (4, (1 << 19) + 1), (1 << 33, 1000)):
        assert size(*bad) == 0
    for fp32 in (False, True):
        sizes = [size(M, 131072, 20, fp32) for M in (0, 1, 3, 16, 17, 100, 127, 128, 129, 513, 4000)]
        assert sizes == sorted(sizes) and sizes[0] > 0


# ---------------------------------------------------------------------------
# binding
# ---------------------------------------------------------------------------

def test_binding_refuses_host_tensors():
    import torch
    moe = _moe()
    bf = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.zeros((48, 64), dtype=torch.bfloat16)
    tok, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    for call in (lambda: moe.moe_linear_gated(bf, w),
                 lambda: moe.moe_linear_gated_backward(bf, w, bf),
                 lambda: moe.moe_linear_adapters(bf, dict(a=w.view(3, 16, 64), b=w.view(3, 64, 16)),
                                                 tok),
                 lambda: moe.moe_token_logprobs(f.view(2, 2), tok),
                 lambda: moe.moe_token_logprobs_backward(f.view(2, 2), tok, f, f, f)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        moe.moe_token_logprobs(bf.half(), tok)
    for make in (lambda: moe.linear_gated_backward_workspace(4, 60, 24),
                 lambda: moe.linear_adapters_workspace(4, 64, 12),
                 lambda: moe.token_logprobs_workspace(4, 20, 21)):
        with pytest.raises(moe.MoeError):
            make()
