"""Argument checks of the scored-routing and dense 4-bit calls on the CPU:
every call here is rejected, or has nothing to do, before any launch."""

from __future__ import annotations

import ctypes

import pytest

NULL = None
FAKE = 0x10000      # never dereferenced
ODD = 0x10004       # not 16-byte aligned


def _moe():
    import mixture_experts_ffn_renorm_amd as moe
    return moe


def rule(score=1, top_k=8, renormalize=1, n_group=8, topk_group=4, group_top=2, scale=2.5,
         bias=None):
    return _moe().RoutingRule(score, top_k, renormalize, n_group, topk_group, group_top, scale, bias)


RULES = [
    (dict(score=2), 256, -1),
    (dict(score=-1), 256, -1),
    (dict(renormalize=2), 256, -1),
    (dict(top_k=0), 256, -1),
    (dict(top_k=40, topk_group=8), 256, -2),
    (dict(n_group=0), 256, -1),
    (dict(n_group=7), 256, -1),                               # does not divide E
    (dict(topk_group=0), 256, -1),
    (dict(topk_group=9), 256, -1),
    (dict(group_top=0), 256, -1),
    (dict(group_top=3), 256, -1),
    (dict(n_group=64, topk_group=8, group_top=2), 64, -1),    # two of one expert
    (dict(topk_group=1, top_k=33, n_group=8), 256, -2),
    (dict(topk_group=1, top_k=5, n_group=8, group_top=1), 32, -1),   # 4 experts stay, 5 are wanted
    (dict(n_group=128, topk_group=8, group_top=1), 256, -2),
    (dict(scale=float("nan")), 256, -1),
    (dict(scale=float("inf")), 256, -1),
    (dict(), 600, -2),
    (dict(), 0, -1),
    (dict(top_k=20, n_group=1, topk_group=1, group_top=1), 16, -1),
]


@pytest.mark.parametrize("change,E,status", RULES)
def test_rules_that_are_refused(change, E, status):
    moe = _moe()
    lib = moe.library()
    r = ctypes.addressof(c := rule(**change))
    assert lib.moe_select(FAKE, r, 4, E, FAKE, FAKE, NULL) == status
    assert lib.moe_select_backward(FAKE, FAKE, FAKE, r, 4, E, FAKE, NULL) == status
    assert lib.moe_route_scored(FAKE, FAKE, NULL, r, 4, 64, E, FAKE, FAKE, FAKE, NULL, 0,
                                NULL) == status
    info = moe.DispatchInfo()
    assert lib.moe_forward_scored(FAKE, FAKE, NULL, r, FAKE, FAKE, 4, E, 128, 128, FAKE, NULL, NULL,
                                  FAKE, 1 << 40, info, NULL) == status
    qw = moe.QuantizedWeights(4, 64, *([FAKE] * 6))
    assert lib.moe_forward_quantized_scored(FAKE, FAKE, NULL, r, qw, 4, E, 128, 128, FAKE, NULL,
                                            NULL, FAKE, 1 << 40, info, NULL) == status
    mw = moe.MxWeights(*([FAKE] * 4))
    assert lib.moe_forward_mxfp8_scored(FAKE, FAKE, NULL, r, mw, 4, E, 128, 128, FAKE, NULL, NULL,
                                        FAKE, 1 << 40, info, NULL) == status
    del c


def test_select_pointers_and_empty_batches():
    lib = _moe().library()
    c = rule()
    r = ctypes.addressof(c)
    assert lib.moe_select(NULL, r, 0, 256, NULL, NULL, NULL) == 0
    assert lib.moe_select_backward(NULL, NULL, NULL, r, 0, 256, NULL, NULL) == 0
    assert lib.moe_route_scored(NULL, NULL, NULL, r, 0, 64, 256, NULL, NULL, NULL, NULL, 0, NULL) == 0
    assert lib.moe_select(FAKE, NULL, 4, 256, FAKE, FAKE, NULL) == -1
    assert lib.moe_select_backward(FAKE, FAKE, FAKE, NULL, 4, 256, FAKE, NULL) == -1
    assert lib.moe_select(FAKE, r, -1, 256, FAKE, FAKE, NULL) == -1
    assert lib.moe_select(FAKE, r, 1 << 22, 256, FAKE, FAKE, NULL) == -2     # M * top_k
    for at in range(3):
        p = [FAKE] * 3
        p[at] = NULL
        assert lib.moe_select(p[0], r, 4, 256, p[1], p[2], NULL) == -1
    assert lib.moe_select(ODD, r, 4, 256, FAKE, FAKE, NULL) == -1
    for at in range(4):
        p = [FAKE] * 4
        p[at] = NULL
        assert lib.moe_select_backward(p[0], p[1], p[2], r, 4, 256, p[3], NULL) == -1
    assert lib.moe_select_backward(ODD, FAKE, FAKE, r, 4, 256, FAKE, NULL) == -1
    assert lib.moe_select_backward(FAKE, FAKE, FAKE, r, 4, 256, ODD, NULL) == -1
    assert lib.moe_select_backward(FAKE, FAKE, FAKE, r, 4, 256, FAKE, NULL) == -1   # in place


def test_route_scored_workspace():
    lib = _moe().library()
    c = rule()
    r = ctypes.addressof(c)
    assert lib.moe_route_scored(FAKE, FAKE, NULL, r, 4, 64, 256, FAKE, FAKE, NULL, NULL, 0, NULL) == -3
    assert lib.moe_route_scored(FAKE, FAKE, NULL, r, 4, 64, 256, FAKE, FAKE, NULL, FAKE,
                                4 * 256 * 4 - 1, NULL) == -3
    assert lib.moe_route_scored(FAKE, FAKE, NULL, r, 4, 60, 256, FAKE, FAKE, FAKE, NULL, 0, NULL) == -2
    assert lib.moe_route_scored(ODD, FAKE, NULL, r, 4, 64, 256, FAKE, FAKE, FAKE, NULL, 0, NULL) == -1


def test_layers_need_a_rule_and_a_workspace():
    moe = _moe()
    lib = moe.library()
    info = moe.DispatchInfo()
    args = (4, 256, 128, 128, FAKE, NULL, NULL, FAKE, 64, info, NULL)
    qw = moe.QuantizedWeights(4, 64, *([FAKE] * 6))
    mw = moe.MxWeights(*([FAKE] * 4))
    assert lib.moe_forward_scored(FAKE, FAKE, NULL, NULL, FAKE, FAKE, *args) == -1
    assert lib.moe_forward_quantized_scored(FAKE, FAKE, NULL, NULL, qw, *args) == -1
    assert lib.moe_forward_mxfp8_scored(FAKE, FAKE, NULL, NULL, mw, *args) == -1
    c = rule()
    r = ctypes.addressof(c)
    assert lib.moe_forward_scored(FAKE, FAKE, NULL, r, FAKE, FAKE, *args) == -3
    # router, selection, one launch of lists, GEMM 1, GEMM 2 and its sum
    info.launches = 0
    assert lib.moe_forward_scored(FAKE, FAKE, NULL, r, FAKE, FAKE, 64, *args[1:]) == -3
    assert info.launches == 6 and info.sorted == 1
    assert lib.moe_forward_quantized_scored(FAKE, FAKE, NULL, r, qw, *args) == -3
    assert lib.moe_forward_mxfp8_scored(FAKE, FAKE, NULL, r, mw, *args) == -3


LINEAR = [
    (dict(out=FAKE), -1),     # x in place
    (dict(bits=8), -2), (dict(group=16), -2), (dict(group=256), -2), (dict(K=96), -2),
    (dict(M=-1), -1), (dict(N=0), -1), (dict(K=0), -1), (dict(gated=2), -1),
    (dict(gated=1, N=33), -1), (dict(M=1 << 24), -2), (dict(N=1 << 24), -2),
    (dict(K=1 << 24), -2), (dict(M=1 << 20, N=1 << 20), -2), (dict(M=0, x=NULL, out=NULL), 0), (dict(x=NULL), -1),
    (dict(out=NULL), -1), (dict(x=ODD), -1), (dict(out=ODD), -1), (dict(addend=ODD), -1),
    (dict(q=NULL), -1), (dict(scales=NULL), -1), (dict(biases=NULL), -1), (dict(q=ODD), -1),
]


@pytest.mark.parametrize("change,status", LINEAR)
def test_linear_refusals(change, status):
    moe = _moe()
    a = dict(x=FAKE, bits=4, group=64, q=FAKE, scales=FAKE, biases=FAKE, M=4, N=32, K=128, gated=0,
             row_scale=NULL, addend=NULL, out=2 * FAKE)
    a.update(change)
    w = moe.QuantizedMatrix(a["bits"], a["group"], a["q"], a["scales"], a["biases"])
    assert moe.library().moe_linear_quantized(
        a["x"], ctypes.addressof(w), a["M"], a["N"], a["K"], a["gated"], a["row_scale"],
        a["addend"], a["out"], NULL) == status
    assert moe.library().moe_linear_quantized(FAKE, NULL, 4, 32, 128, 0, NULL, NULL, FAKE, NULL) == -1


def test_binding_refuses_host_tensors_and_bad_rules():
    import torch
    moe = _moe()
    with pytest.raises(ValueError):
        moe.Routing(2, score="tanh")
    with pytest.raises(ValueError):
        moe.Routing(2, select_bias=torch.zeros(4))
    r = moe.Routing(2, score="sigmoid", n_group=4, scale=2.0)
    assert (r.top_k, r.score, r.renormalize, r.n_group, r.topk_group, r.group_top, r.scale) == \
        (2, "sigmoid", True, 4, 4, 1, 2.0)
    with pytest.raises(ValueError):
        moe.moe_select(torch.zeros(3, 4), r)
    with pytest.raises(ValueError):
        moe.moe_select_backward(torch.zeros(3, 4), torch.zeros(3, 2), torch.zeros(3, 2), r)
    w = dict(bits=4, group_size=64, q=torch.zeros(8, 8, dtype=torch.int32),
             scales=torch.zeros(8, 1, dtype=torch.bfloat16),
             biases=torch.zeros(8, 1, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        moe.moe_linear_quantized(torch.zeros(3, 64, dtype=torch.bfloat16), w)
    with pytest.raises(moe.MoeError):
        moe.moe_linear_quantized(torch.zeros(3, 64, dtype=torch.bfloat16), dict(w, bits=8))


def test_misaligned_bias():
    lib = _moe().library()
    c = rule(bias=ODD)
    assert lib.moe_select(FAKE, ctypes.addressof(c), 4, 256, FAKE, FAKE, NULL) == -1


def test_packed_matrix_is_the_struct():
    moe = _moe()
    w = moe.QuantizedMatrix(4, 64, 0x1230, 0x4560, 0x7890)
    assert moe._pack_matrix(4, 64, 0x1230, 0x4560, 0x7890) == bytes(w)
