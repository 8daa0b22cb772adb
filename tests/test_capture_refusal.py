"""The rule that refuses a captured backward pass whose leaves belong to an
autograd graph from before the capture.  On the CPU: the nodes and streams are
plain values here, and nothing is captured."""

import pytest
import torch

from mxfp8_block_scaled_amd import api


def test_leaf_of_a_living_graph_on_another_stream():
    x, w = (torch.ones(3, requires_grad=True) for _ in range(2))
    eager = x * w
    api._mark_leaves(eager, 0)
    captured = x * w
    api._mark_leaves(captured, 7)
    api._check_capture(captured.grad_fn, 7, capturing=False)
    with pytest.raises(RuntimeError, match="alive on another stream"):
        api._check_capture(captured.grad_fn, 7, capturing=True)
    # the same stream is no obstacle
    api._check_capture(captured.grad_fn, 0, capturing=True)
    # one operand of the old graph is enough
    other = torch.ones(3, requires_grad=True)
    mixed = other * w
    api._mark_leaves(mixed, 7)
    with pytest.raises(RuntimeError, match="alive on another stream"):
        api._check_capture(mixed.grad_fn, 7, capturing=True)


def test_leaf_whose_graph_is_gone_and_computed_operands():
    x, w = (torch.ones(3, requires_grad=True) for _ in range(2))
    eager = x * w
    api._mark_leaves(eager, 0)
    del eager
    captured = (x * 1.0) * w
    api._mark_leaves(captured, 7)
    api._check_capture(captured.grad_fn, 7, capturing=True)
    # operands without gradients
    half = x * torch.ones(3)
    api._mark_leaves(half, 7)
    api._check_capture(half.grad_fn, 7, capturing=True)
