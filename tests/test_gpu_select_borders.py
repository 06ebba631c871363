"""Scored routing where a plain fp32 evaluation goes wrong: masks of the type's lowest value."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import moe_oracle as mo
from tests import helpers as h
from tests import test_gpu_select as ts

pytestmark = pytest.mark.gpu

INF = np.float32(np.inf)
LOWEST = np.finfo(np.float32).min


@pytest.mark.parametrize("low", [-INF, LOWEST, np.float32(-1e9)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_group_sums_with_masking_biases(score, low):
    """Biases that mask experts: one expert left in some groups, none in
    others, a group's sum past the type's lowest value."""
    E, G = 96, 8
    l = ts.draw(300, E, 17)
    bias = ts.steps(E, 18)
    bias[1:12] = low                        # one expert of group 0 stays
    bias[12:24] = low                       # none of group 1
    bias[24:35] = low
    bias[40:44] = low
    for kept in (1, 3, 6, 7, 8):
        for top in (1, 2):
            ts.check(l, 8 if kept > 1 else 2, score, True, bias, G, kept, top)


@pytest.mark.parametrize("low", [-INF, LOWEST, np.float32(-1e9)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,M", [(33, 1, 9), (60, 1, 4000), (510, 1, 700), (510, 5, 9), (3, 1, 5)])
def test_masking_biases_where_lanes_have_spare_experts(E, G, M, score, low):
    """The choice reaches masked experts, and lanes hold places for experts
    that do not exist: those are never chosen."""
    bias = ts.steps(E, 19)
    bias[2:E // G] = low
    if G > 1:
        bias[E // G:] = low
    l = ts.draw(M, E, 20)
    k = min(E, 6)
    ids, _ = ts.check(l, k, score, True, bias, G, min(G, 2), 1)
    assert np.all((ids >= 0) & (ids < E))
