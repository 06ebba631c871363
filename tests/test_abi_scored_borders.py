"""Calls of scored routing and dense 4-bit products that are refused before any
launch: operands that overlap, sizes that the C interface cannot hold."""

from __future__ import annotations

import ctypes

import pytest

from tests.test_abi_scored import NULL, _moe, rule

A = 0x1000000       # never dereferenced
STEP = 0x100000     # more than any operand here


def select(lib, r, **at):
    """moe_select of 4 tokens, 256 experts, top_k 8 with the given pointers."""
    p = dict(logits=A, ids=A + STEP, weights=A + 2 * STEP)
    p.update(at)
    return lib.moe_select(p["logits"], r, 4, 256, p["ids"], p["weights"], NULL)


def test_select_outputs_that_overlap():
    lib = _moe().library()
    c = rule(bias=A + 4 * STEP)
    r = ctypes.addressof(c)
    logits, pairs = 4 * 256 * 4, 4 * 8 * 4
    for at in (dict(ids=A), dict(weights=A), dict(ids=A + logits - 4), dict(weights=A - pairs + 4),
               dict(weights=A + STEP), dict(weights=A + STEP + pairs - 4),
               dict(ids=A + 4 * STEP + 16), dict(weights=A + 4 * STEP + 256 * 4 - 4)):
        assert select(lib, r, **at) == -1, at


def backward(lib, r, **at):
    p = dict(logits=A, ids=A + STEP, grad=A + 2 * STEP, out=A + 3 * STEP)
    p.update(at)
    return lib.moe_select_backward(p["logits"], p["ids"], p["grad"], r, 4, 256, p["out"], NULL)


def test_gradient_that_overlaps_an_operand():
    lib = _moe().library()
    c = rule()
    r = ctypes.addressof(c)
    logits, pairs = 4 * 256 * 4, 4 * 8 * 4
    for at in (dict(out=A), dict(out=A + logits - 16), dict(out=A - logits + 16),
               dict(out=A + STEP), dict(out=A + STEP + pairs - 16), dict(out=A + 2 * STEP),
               dict(out=A + 2 * STEP - logits + 16)):
        assert backward(lib, r, **at) == -1, at


def linear(lib, moe, M=4, N=32, K=128, group=64, gated=0, row_scale=NULL, addend=NULL, x=A,
           out=A + STEP, q=A + 2 * STEP, s=A + 3 * STEP, b=A + 4 * STEP):
    w = moe.QuantizedMatrix(4, group, q, s, b)
    return lib.moe_linear_quantized(x, ctypes.addressof(w), M, N, K, gated, row_scale, addend, out,
                                    NULL)


def test_product_that_overlaps_an_operand():
    moe = _moe()
    lib = moe.library()
    x, out = 4 * 128 * 2, 4 * 32 * 2
    for at in (dict(out=A), dict(out=A + x - 16), dict(out=A - out + 16),
               dict(addend=A + STEP + 16), dict(addend=A + STEP - out + 16),
               dict(row_scale=A + STEP + out - 4), dict(row_scale=A + STEP - 12),
               dict(q=A + STEP + out - 16), dict(s=A + STEP), dict(b=A + STEP - 112),
               dict(gated=1, out=A + x - 16), dict(gated=1, addend=A + STEP + out // 2 - 16)):
        assert linear(lib, moe, **at) == -1, at


@pytest.mark.parametrize("field", ["top_k", "n_group", "topk_group", "group_top"])
@pytest.mark.parametrize("value", [2 ** 32 + 1, 2 ** 31, -2 ** 31 - 1, 2 ** 64 + 2])
def test_rule_numbers_beyond_the_struct(field, value):
    """A number that a C int cannot hold is refused, not cut to its low bits."""
    moe = _moe()
    with pytest.raises(ValueError):
        moe.Routing(**{"top_k": 2, field: value})


def test_sizes_beyond_the_interface():
    """A dimension that a C int cannot hold is refused before anything else,
    not cut to its low bits."""
    import torch
    moe = _moe()
    big = 2 ** 32 + 5

    def meta(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="meta")

    bf16, r = torch.bfloat16, moe.Routing(1, score="sigmoid")
    with pytest.raises(moe.MoeError):
        moe.moe_select(meta(big, 1), r)
    with pytest.raises(moe.MoeError):
        moe.moe_select(meta(1, big), r)
    with pytest.raises(moe.MoeError):
        moe.moe_select_backward(meta(big, 1), meta(big, 1, dtype=torch.int32), meta(big, 1), r)
    with pytest.raises(moe.MoeError):
        moe.moe_route_scored(meta(big, 8, dtype=bf16), meta(1, 8, dtype=bf16), r)
    with pytest.raises(moe.MoeError):
        moe.moe_route_scored(meta(1, big + 3, dtype=bf16), meta(1, big + 3, dtype=bf16), r)

    def matrix(N, K):
        return dict(bits=4, group_size=64, q=meta(N, K // 8, dtype=torch.int32),
                    scales=meta(N, K // 64, dtype=bf16), biases=meta(N, K // 64, dtype=bf16))

    for M, N, K in ((big, 8, 64), (1, big, 64), (1, 8, 2 ** 32 + 64)):
        with pytest.raises(moe.MoeError):
            moe.moe_linear_quantized(meta(M, K, dtype=bf16), matrix(N, K))
    w13, w2 = meta(1, 16, 8, dtype=bf16), meta(1, 8, 8, dtype=bf16)
    with pytest.raises(moe.MoeError):
        moe.moe_forward_scored(meta(big, 8, dtype=bf16), meta(1, 8, dtype=bf16), w13, w2, r)
