"""What a program may do with the outputs of moe_token_logprobs."""

from __future__ import annotations

import pytest

from tests import test_gpu_logprobs as tl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 5])
@pytest.mark.parametrize("top", [0, 3])
def test_outputs_are_tensors_of_their_own(M, top):
    """A change of one, also under autograd, is no change of another."""
    import torch
    moe = tl._moe()
    l, _ = tl.device(tl.draw(M, 1000, M), "float32")
    tok = torch.arange(M, dtype=torch.int32, device="cuda")
    fresh = moe.moe_token_logprobs(l, tok, top=top)[:3]
    for k in range(3):
        outs = moe.moe_token_logprobs(l, tok, top=top)[:3]
        rest = [t for i, t in enumerate(outs) if i != k]
        before = [t._version for t in rest]
        weight = torch.full((M,), 2.0, device="cuda", requires_grad=True)
        outs[k].mul_(weight)
        assert outs[k].requires_grad and [t._version for t in rest] == before
        assert not any(t.requires_grad for t in rest)
        outs[k].sum().backward()
        assert torch.equal(weight.grad, fresh[k])
        assert all(torch.equal(t, f) for t, f in zip(rest, (f for i, f in enumerate(fresh) if i != k)))
