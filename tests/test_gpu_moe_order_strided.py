"""moe_permute and moe_unpermute on leaves that have to be laid out anew, eager and captured."""

import pytest
import torch

from mxfp8_block_scaled_amd import api
from tests import gpu_util
from tests.test_gpu_moe_order import make_ids

pytestmark = pytest.mark.gpu
dev = gpu_util.dev
T, TOPK, E, H = 90, 3, 7, 70


def operands():
    g = torch.Generator(device=dev()).manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, device=dev())
    return n(H, T).t(), n(H, T * TOPK).t(), n(TOPK, T).t(), n(H, T * TOPK).t(), n(H, T).t()


def step(x, ys, w, order, dxs, dy):
    return torch.autograd.grad((api.moe_permute(x, order), api.moe_unpermute(ys, order, w)), (x, ys, w), (dxs, dy))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients(dtype):
    order = api.moe_sort(make_ids(T, TOPK, E, 1, 0.2).to(dev()), E)
    x, ys, w, dxs, dy = operands()
    a = [t.to(dtype) for t in (x, ys)] + [w] + [t.to(dtype) for t in (dxs, dy)]
    assert not any(t.is_contiguous() for t in a)
    turned = step(*(t.detach().requires_grad_() for t in a[:3]), order, *a[3:])
    plain = step(*(t.contiguous().requires_grad_() for t in a[:3]), order, *(t.contiguous() for t in a[3:]))
    for u, v in zip(turned, plain):
        assert u.shape == v.shape and torch.equal(u, v)


def test_captured():
    order = api.moe_sort(make_ids(T, TOPK, E, 2, 0.2).to(dev()), E)
    x, ys, w, dxs, dy = operands()
    leaves = [t.detach().requires_grad_() for t in (x, ys, w)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*leaves, order, dxs, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(*leaves, order, dxs, dy)
    for _ in range(3):
        for t in (x, ys, w, dxs, dy):
            t.add_(0.5)
        graph.replay()
        want = step(*(t.detach().clone().requires_grad_() for t in (x, ys, w)), order, dxs, dy)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("which", ["x", "ys", "w"])
def test_capture_with_a_live_eager_graph_is_refused(which):
    order = api.moe_sort(make_ids(T, TOPK, E, 3).to(dev()), E)
    x, ys, w, _, _ = operands()
    if which == "x":
        x.requires_grad_()
        call = lambda: api.moe_permute(x, order)
    else:
        (ys if which == "ys" else w).requires_grad_()
        call = lambda: api.moe_unpermute(ys, order, w)
    alive = call()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="captured"):
        with torch.cuda.graph(graph):
            call().sum().backward()
    torch.cuda.synchronize()
    assert alive.requires_grad
