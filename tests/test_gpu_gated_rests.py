"""The bf16 gated block where the last round of tiles leaves few rows, which
become a product of their own, and gradients of few features."""

from __future__ import annotations

import pytest

from tests import helpers as h
from tests import test_gpu_gated as tg

pytestmark = pytest.mark.gpu

# 256 x 256 tiles: 8 rows of them are whole rounds of the chip, the rest is left
RESTS = [2049, 2050, 2064, 2065, 2080, 2112]


@pytest.mark.parametrize("M", RESTS)
def test_rests(M):
    tg.check(M, 64, 4096, M)


@pytest.mark.parametrize("M", RESTS)
def test_gradient_rests(M):
    tg.check_grad(M, 64, 4096, M)


@pytest.mark.parametrize("M", [2049, 2064, 2065])
def test_gradient_writes_no_row_behind_the_last(M):
    """d_gate and d_up are M rows of the workspace.  grad_w13 of 64 x 4 tiles is
    cut into no ranges, so what lies behind them stays as it was."""
    import torch
    H, I = 512, 4096
    moe = tg._moe()
    x, w, d = (h.dev_bf16(t) for t in tg.inputs(M, H, I, M))
    ws = torch.full((moe.moe_linear_gated_backward_workspace_size(M, H, I),), 255,
                    dtype=torch.uint8, device="cuda")
    _, gw = moe.moe_linear_gated_backward(x, w, d, need_x=False, ws=ws)
    torch.cuda.synchronize()
    used = (M * 2 * I * 2 + 255) // 256 * 256
    assert 0 < used < ws.numel()
    assert (ws[used:] == 255).all()
    # the rows themselves: a NaN left among them would reach every feature
    assert torch.isfinite(gw).all()


@pytest.mark.parametrize("M,H,I", [(1000, 2048, 200), (1024, 2048, 64), (1030, 2048, 200),
                                   (300, 8192, 248), (700, 4096, 496), (2100, 2048, 248),
                                   (4099, 2048, 256), (1100, 8200, 104)])
def test_gradient_of_few_features(M, H, I):
    """grad_x whose sums are short, its tiles on both sides of half the chip."""
    tg.check_grad(M, H, I, M, need=(True, False))
