"""The dense operators one after another, as a training or scoring step runs
them: a gated block, a 4-bit head with the requests' adapters, log
probabilities, their gradient in place of the logits, and the block's gradient;
all through one workspace, eagerly and as a replayed graph."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import dense_oracle as do
from oracle import moe_oracle as mo
from tests import helpers as h
from tests import test_gpu_adapters as ta
from tests import test_gpu_gated as tg
from tests import test_gpu_logprobs as tl
from tests import test_gpu_qlinear as ql

pytestmark = pytest.mark.gpu


def host_bits(t):
    import torch
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("M", [1, 60, 300])
def test_a_step(M):
    import torch
    import mixture_experts_ffn_renorm_amd as moe
    H, I, V, S, R, group, top = 256, 128, 2000, 6, 16, 64, 4
    x, w13, _ = tg.inputs(M, H, I, M)
    head = ql.matrix(V, I, group, 5)
    ad = ta.inputs(M, S, R, I, V, M + 1)
    dx, dw = h.dev_bf16(x), h.dev_bf16(w13)
    dhead = ql.to_device(*head, group)
    dad = dict(a=h.dev_bf16(ad["a"]), b=h.dev_bf16(ad["b"]), scales=h.dev_f32(ad["scales"]))
    slots = h.dev_i32(ad["random"])
    tokens = h.dev_i32(np.random.default_rng(2).integers(0, V, M))
    rng = np.random.default_rng(3)
    g, e = (rng.standard_normal(M).astype(np.float32) for _ in range(2))
    dg, de = h.dev_f32(g), h.dev_f32(e)
    # the head's rows as numbers, for the product that is not under test
    wide = torch.from_numpy(dequantized(head, group)).cuda()
    ws = torch.empty(max(moe.moe_linear_gated_backward_workspace_size(M, H, I),
                         moe.moe_linear_adapters_workspace_size(M, I, R),
                         moe.moe_token_logprobs_workspace_size(M, V, top)),
                     dtype=torch.uint8, device="cuda")

    def step():
        act = moe.moe_linear_gated(dx, dw)
        shared = moe.moe_linear_quantized(act, dhead)
        logits = moe.moe_linear_adapters(act, dad, slots, addend=shared, ws=ws)
        lp, ent, lse, ids, tlp = moe.moe_token_logprobs(logits, tokens, top=top, ws=ws)
        grad = moe.moe_token_logprobs_backward(logits, tokens, lse, ent, dg, de,
                                               grad_logits=logits.clone())
        d_act = (grad.float() @ wide).to(torch.bfloat16)
        gx, gw = moe.moe_linear_gated_backward(dx, dw, d_act, ws=ws)
        return act, shared, logits, lp, ent, lse, ids, tlp, grad, d_act, gx, gw

    out = step()
    torch.cuda.synchronize()
    act, shared, logits, lp, ent, lse, ids, tlp, grad, d_act, gx, gw = out

    # each step from the bits that the one before left
    X, W, gate, up, eg, eu = tg.parts(x, w13)
    assert np.all(np.abs(h.host_bf16_to_f64(act) - do.gated(X, W)) <= tg.act_bound(gate, up, eg, eu))
    a_bits = host_bits(act)
    ref = mo.linear_quantized(a_bits, *head, group)
    bound = ql.error_bound(a_bits, *head, group, False, None, None)
    assert np.all(np.abs(h.host_bf16_to_f64(shared) - ref) <= bound + (np.abs(ref) + bound) * ta.B)
    ref, bound = ta.reference(dict(ad, x=a_bits, addend=host_bits(shared)), ad["random"], True, True,
                              False)
    assert np.all(np.abs(h.host_bf16_to_f64(logits) - ref) <= bound)
    l = logits.float().cpu().numpy()
    tok = tokens.cpu().numpy()
    want = do.token_logprobs(l, tok, top)
    el, ee, ep = tl.bounds(l)
    tl.compare("logprobs", lp.cpu().numpy(), want["logprobs"], ep + 3 * tl.U * np.abs(want["logprobs"]))
    tl.compare("entropy", ent.cpu().numpy(), want["entropy"], ee)
    tl.compare("lse", lse.cpu().numpy(), want["lse"], el)
    assert np.array_equal(ids.cpu().numpy(), want["top_ids"])
    ref = do.token_logprobs_backward(l, tok, lse.cpu().numpy(), ent.cpu().numpy(), g, e)
    tl.compare("grad", grad.double().cpu().numpy(), ref,
               tl.grad_bound(l, lse.cpu().numpy(), ent.cpu().numpy(), g, e, ref, "bfloat16"))
    d_bits = host_bits(d_act)
    want = do.gated_backward(X, W, mo.widen_bf16(d_bits).astype(np.float64))
    for got, ref, (_, bound) in zip((gx, gw), want, tg.grad_bounds(x, w13, d_bits)):
        assert np.all(np.abs(h.host_bf16_to_f64(got) - ref) <= bound)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = step()
    for _ in range(3):
        for t in again:
            t.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, out))


def dequantized(head, group):
    """[V, K] fp32 of the head's codes: w = s q + b."""
    q, s, b = head
    codes = (q[:, :, None] >> (4 * np.arange(8, dtype=np.uint32))) & 15
    V = q.shape[0]
    codes = codes.reshape(V, -1, group).astype(np.float64)
    w = codes * mo.widen_bf16(s)[:, :, None] + mo.widen_bf16(b)[:, :, None]
    return w.reshape(V, -1).astype(np.float32)
