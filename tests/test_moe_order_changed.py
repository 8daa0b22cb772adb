"""An order that is changed in place between forward and backward pass: refused, as torch refuses it for tensors that an
operator has saved.  On the CPU, with a stand-in for the library."""

import pytest
import torch

from mxfp8_block_scaled_amd import api

T, TOPK, H = 4, 2, 6


class Library:
    """Backward calls that succeed and write nothing."""

    def __getattr__(self, name):
        return lambda *args: 0


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    monkeypatch.setattr(api, "_stream", lambda device=None: 0)
    monkeypatch.setattr(api, "_require_cuda", lambda t, name: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(api, "lib", lambda: Library())


def order():
    return api.MoEOrder(torch.arange(T * TOPK, dtype=torch.int32).view(T, TOPK),
                        torch.arange(T * TOPK, dtype=torch.int32), torch.tensor([0, 4, 8, 8], dtype=torch.int32))


def outputs(o):
    x, ys, w = (torch.ones(*s, requires_grad=True) for s in ((T, H), (T * TOPK, H), (T, TOPK)))
    return (api.moe_permute(x, o), api.moe_unpermute(ys, o, w), api.moe_unpermute(ys, o),
            api.moe_unpermute(ys.detach(), o, w))


@pytest.mark.parametrize("which", ["rows", "offsets"])
@pytest.mark.parametrize("out", range(4))
def test_changed_in_place(which, out):
    o = order()
    y = outputs(o)[out]
    getattr(o, which).add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("out", range(4))
def test_unchanged(out):
    o = order()
    y = outputs(o)[out]
    o.slots.add_(1)                  # which no gradient reads
    y.sum().backward(retain_graph=True)
    y.sum().backward()


@pytest.mark.parametrize("which", ["rows", "offsets"])
@pytest.mark.parametrize("out", range(4))
def test_replaced(which, out):
    o = order()
    y = outputs(o)[out]
    setattr(o, which, getattr(o, which).clone())
    with pytest.raises(RuntimeError, match="replaced"):
        y.sum().backward()


def test_permutes_gradient_needs_no_retained_graph():
    x, o = torch.ones(T, H, requires_grad=True), order()
    xs = api.moe_permute(x, o)
    for _ in range(2):
        torch.autograd.grad(xs, x, torch.ones_like(xs))


def test_made_in_inference_mode():
    """Its tensors have no version, and may be used all the same."""
    with torch.inference_mode():
        o = order()
    for y in outputs(o):
        y.sum().backward()
