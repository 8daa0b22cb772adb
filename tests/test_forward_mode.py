"""The operators with gradients are differentiable in reverse mode only: an operand that carries a tangent of
torch.autograd.forward_ad is refused, not taken without it.  On the CPU for the calls that no reverse gradient is asked
of, which go past the autograd node; those of a node are refused by torch, behind the kernels."""

import pytest
import torch
from torch.autograd import forward_ad

from mxfp8_block_scaled_amd import api


def calls(device):
    """(call of one operand, that operand) for every operand with a gradient."""
    n = lambda *s, dtype=torch.float32: torch.ones(*s, dtype=dtype, device=device)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=device)
    order = api.MoEOrder(i(4, 2), i(8), i(4))
    x, ys, w = n(4, 6), n(8, 6), n(4, 2)
    a, b, c = (n(*s, dtype=torch.bfloat16) for s in ((4, 16), (16, 16), (16,)))
    return {
        "permute": (lambda t: api.moe_permute(t, order), x),
        "unpermute rows": (lambda t: api.moe_unpermute(t, order, w), ys),
        "unpermute weights": (lambda t: api.moe_unpermute(ys, order, t), w),
        "linear_b128 x": (lambda t: api.linear_b128(t, b, c), a),
        "linear_b128 w": (lambda t: api.linear_b128(a, t, c), b),
        "linear_b128 bias": (lambda t: api.linear_b128(a, b, t), c),
        "balance": (lambda t: api.moe_balance_loss(t, 2), n(4, 6)),
    }


class Reached(Exception):
    pass


@pytest.mark.parametrize("name", sorted(set(calls("cpu")) - {"balance"}))   # (the loss has no way past its node)
@pytest.mark.parametrize("requires_grad,grad", [(False, False), (False, True), (True, False)])
def test_past_the_node(name, requires_grad, grad, monkeypatch):
    def kernels(*args):
        raise Reached
    monkeypatch.setattr(api, "_require_cuda", lambda t, name: None)
    for f in ("_permute", "_unpermute", "_linear_b128_forward"):
        monkeypatch.setattr(api, f, kernels)
    call, t = calls("cpu")[name]
    with torch.set_grad_enabled(grad):
        with forward_ad.dual_level():
            dual = forward_ad.make_dual(t.detach().requires_grad_(requires_grad), torch.ones_like(t))
            with pytest.raises(RuntimeError, match="reverse mode"):
                call(dual)
            # without a tangent: as outside of the level
            with pytest.raises(Reached):
                call(t)
        with pytest.raises(Reached):
            call(t)


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(calls("cpu")))
@pytest.mark.parametrize("requires_grad", [False, True])
@pytest.mark.parametrize("grad", [False, True])
def test_every_operand(name, requires_grad, grad):
    call, t = calls("cuda")[name]
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        dual = forward_ad.make_dual(t.detach().requires_grad_(requires_grad), torch.ones_like(t))
        with pytest.raises(RuntimeError, match="reverse mode|jvp"):
            call(dual)
        call(t)
    torch.cuda.synchronize()
