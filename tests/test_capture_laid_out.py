"""Captured backward passes of moe_permute and moe_unpermute whose operands have to be laid out anew (rows that are not
contiguous, strided weights): a leaf among them is as visible to the rule that refuses a capture as any other.  On the
CPU: streams are plain values, the kernels stand-ins, and nothing is captured."""

import pytest
import torch

from mxfp8_block_scaled_amd import api

T, TOPK, E, H = 4, 2, 3, 6


class Streams:
    now, capturing = 0, False


@pytest.fixture
def streams(monkeypatch):
    s = Streams()
    monkeypatch.setattr(api, "_stream", lambda device=None: s.now)
    monkeypatch.setattr(api, "_require_cuda", lambda t, name: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: s.capturing)

    def laid_out(t):
        assert t.stride(1) == 1 and t.stride(0) >= t.shape[1]
        return t

    def permute(x, order):
        return laid_out(x).repeat_interleave(TOPK, 0)

    def unpermute(ys, order, weights):
        assert weights is None or weights.is_contiguous()
        return laid_out(ys).view(T, TOPK, H).sum(1)

    monkeypatch.setattr(api, "_permute", permute)
    monkeypatch.setattr(api, "_unpermute", unpermute)
    return s


def order():
    return api.MoEOrder(torch.arange(T * TOPK, dtype=torch.int32).view(T, TOPK),
                        torch.arange(T * TOPK, dtype=torch.int32), torch.tensor([0, 4, 8, 8], dtype=torch.int32))


def leaf(rows, turned):
    return torch.ones(H, rows).t().requires_grad_() if turned else torch.ones(rows, H, requires_grad=True)


def weights(turned):
    return torch.ones(TOPK, T).t().requires_grad_() if turned else torch.ones(T, TOPK, requires_grad=True)


@pytest.mark.parametrize("turned", [False, True])
def test_permute(streams, turned):
    o, x = order(), leaf(T, turned)
    alive = api.moe_permute(x, o)
    streams.now, streams.capturing = 7, True
    with pytest.raises(RuntimeError, match="captured"):
        api.moe_permute(x, o).sum().backward()
    del alive
    api.moe_permute(x, o).sum().backward()
    assert torch.equal(x.grad, torch.full((T, H), float(TOPK)))


@pytest.mark.parametrize("turned_ys,turned_w", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("which", ["ys", "weights", "both"])
def test_unpermute(streams, turned_ys, turned_w, which):
    o, ys, w = order(), leaf(T * TOPK, turned_ys), weights(turned_w)
    ys.requires_grad_(which != "weights")
    w.requires_grad_(which != "ys")
    alive = api.moe_unpermute(ys, o, w)
    streams.now, streams.capturing = 7, True
    with pytest.raises(RuntimeError, match="captured"):
        api.moe_unpermute(ys, o, w).sum().backward()
    assert alive.shape == (T, H)


def test_leaves_are_the_nodes_own_operands(streams):
    """No node of another operator between them, which would hide them."""
    o = order()
    for turned in (False, True):
        x, ys, w = leaf(T, turned), leaf(T * TOPK, turned), weights(turned)
        for out, leaves in ((api.moe_permute(x, o), (x,)), (api.moe_unpermute(ys, o, w), (ys, w))):
            found = [getattr(n, "variable", None) for n, _ in out.grad_fn.next_functions if n is not None]
            assert len(found) == len(leaves) and all(a is b for a, b in zip(found, leaves))
