"""Overlaps of operands that the dense operators refuse in calls without rows,
which still write an output."""

from __future__ import annotations

import pytest

from tests import test_abi_dense as td


@pytest.mark.parametrize("inside", [0, 16, 2 * 24 * 64 * 2 - 16])
def test_gradient_without_rows_leaves_the_weights_alone(inside):
    """grad_w13 is set to 0 where there are no rows: not in w13's memory."""
    for other in (dict(x=td.NULL, d=td.NULL, ws=td.NULL, gx=td.NULL), dict()):
        assert td.backward(M=0, gw=td.at(1) + inside, **other) == -1
        assert td.backward(M=0, w=td.at(5) + inside, **other) == -1


def test_gradient_without_rows_or_weights_gradient():
    assert td.backward(M=0, gw=td.NULL) == 0
    assert td.backward(M=0, gw=td.NULL, w=td.NULL) == 0
