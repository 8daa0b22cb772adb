"""The counts that moe_balance_loss returns are the caller's: what becomes of
them changes no gradient.  A collective (torch.distributed.all_reduce, say)
writes into a tensor without autograd's notice, as writing through .data does
here."""

import pytest
import torch

from mxfp8_block_scaled_amd import api

T, E, K = 37, 12, 3


CHANGES = {"without notice": lambda c: c.data.mul_(2), "in place": lambda c: c.mul_(2)}


def use(logits, change):
    """(counts as returned, gradient after the change)"""
    loss, counts = api.moe_balance_loss(logits, K, z_coef=1e-3)
    before = counts.clone()
    change(counts)
    return before, torch.autograd.grad(loss, logits)[0]


def plain_forward(logits, topk, valid=None, coef=1e-2, z_coef=0.0):
    counts = torch.bincount(logits.topk(topk).indices.reshape(-1), minlength=logits.shape[1]).int()
    return logits.logsumexp(1).sum(), counts, torch.tensor([len(logits)], dtype=torch.int32)


def plain_backward(logits, topk, counts, used, valid=None, coef=1e-2, z_coef=0.0, grad=None):
    p = logits.softmax(1)
    return grad * coef * p * (counts - (p * counts).sum(1, keepdim=True)) / used


@pytest.mark.parametrize("change", CHANGES)
def test_host_side(monkeypatch, change):
    """The autograd function alone, around plain forms in the kernels' place."""
    monkeypatch.setattr(api, "moe_balance", plain_forward)
    monkeypatch.setattr(api, "moe_balance_backward", plain_backward)
    monkeypatch.setattr(api, "_stream", lambda device=None: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(0)).requires_grad_()
    want = use(x, lambda c: None)
    for p, q in zip(use(x, CHANGES[change]), want):
        assert torch.equal(p, q)


@pytest.mark.gpu
@pytest.mark.parametrize("change", CHANGES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_kernels(dtype, change):
    from tests.gpu_util import dev
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(1)).to(dtype).to(dev()).requires_grad_()
    _, counts, used = api.moe_balance(x.detach(), K, z_coef=1e-3)
    want = api.moe_balance_backward(x.detach(), K, counts, used, z_coef=1e-3)
    c, g = use(x, CHANGES[change])
    assert torch.equal(c, counts) and torch.equal(g, want)
