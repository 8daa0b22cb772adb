"""Tokens sorted by expert and back against plain 64-bit forms."""

import pytest
import torch

from mxfp8_block_scaled_amd import api
from tests import gpu_util

pytestmark = pytest.mark.gpu
dev = gpu_util.dev


def sort_ref(ids, E):
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    slots = torch.sort(key, stable=True).indices
    rows = torch.empty_like(slots)
    rows[slots] = torch.arange(flat.numel())
    counts = torch.bincount(key, minlength=E + 1)
    return rows.view(ids.shape), slots, torch.cumsum(counts, 0) - counts


def make_ids(T, topk, E, seed, drop=0.0):
    g = torch.Generator().manual_seed(seed)
    skew = torch.rand(T, E, generator=g) * torch.rand(E, generator=g)
    ids = torch.topk(skew, min(topk, E), dim=1).indices
    if topk > E:
        ids = torch.randint(0, E, (T, topk), generator=g)
    return torch.where(torch.rand(ids.shape, generator=g) < drop, torch.full_like(ids, -1), ids)


SORTS = [(1, 1, 1), (1, 8, 128), (3, 2, 5), (64, 1, 64), (65, 3, 7), (511, 8, 128), (512, 8, 256), (513, 8, 128),
         (4096, 8, 128), (10007, 4, 60), (70000, 16, 256), (300000, 1, 3)]


@pytest.mark.parametrize("T,topk,E", SORTS)
@pytest.mark.parametrize("drop", [0.0, 0.3])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(T, topk, E, drop, dtype):
    ids = make_ids(T, topk, E, T + topk, drop)
    order = api.moe_sort(ids.to(dtype).to(dev()), E)
    rows, slots, offsets = sort_ref(ids, E)
    assert torch.equal(order.rows.cpu().long(), rows)
    assert torch.equal(order.slots.cpu().long(), slots)
    assert torch.equal(order.offsets.cpu().long(), offsets)


def test_sort_unusual_ids():
    """All of one expert, none of any, the same expert twice in a token, ids far
    out of range in 64 bits, a strided view."""
    for ids in (torch.full((700, 8), 3), torch.full((700, 8), 99), torch.full((2, 2), -7),
                torch.tensor([[1, 1, 1], [0, 1, 0]]), torch.tensor([[2 ** 32, 1], [-2 ** 40, 2 ** 32 + 1]])):
        order = api.moe_sort(ids.to(dev()), 4)
        rows, slots, offsets = sort_ref(ids, 4)
        assert torch.equal(order.rows.cpu().long(), rows) and torch.equal(order.offsets.cpu().long(), offsets)
        assert torch.equal(order.slots.cpu().long(), slots)
    ids = make_ids(50, 8, 16, 1)
    order = api.moe_sort(ids.to(dev())[:, ::2], 16)
    assert torch.equal(order.rows.cpu().long(), sort_ref(ids[:, ::2], 16)[0])
    order = api.moe_sort(torch.empty(0, 4, dtype=torch.int32, device=dev()), 5)
    assert order.offsets.tolist() == [0] * 6 and order.rows.shape == (0, 4)


ROWS = [(1, 1, 4, 1), (1, 8, 16, 2048), (5, 2, 3, 7), (33, 4, 8, 130), (100, 16, 20, 1003), (2100, 3, 5, 72),
        (2500, 8, 64, 264), (600, 1, 4, 4096)]


def inputs(T, topk, E, H, dtype, seed, drop):
    g = torch.Generator().manual_seed(seed)
    ids = make_ids(T, topk, E, seed, drop)
    n = lambda *s: torch.randn(*s, generator=g)
    return (ids, n(T, H).to(dtype), n(T * topk, H).to(dtype), torch.rand(T, topk, generator=g), n(T * topk, H).to(dtype),
            n(T, H).to(dtype))


def close(got, want, eps, terms, scale):
    """fp32 sums of `terms` products of at most `scale` in total magnitude, then a rounding to got's type."""
    err = (got.double().cpu() - want).abs()
    tol = eps / 2 * want.abs() + (1 + eps) * terms * 2.0 ** -23 * scale + 1e-38
    assert bool((err <= tol).all()), (float((err - tol).max()), int((err > tol).sum()))


@pytest.mark.parametrize("T,topk,E,H", ROWS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drop", [0.0, 0.4])
@pytest.mark.parametrize("weighted", [True, False])
def test_there_and_back(T, topk, E, H, dtype, drop, weighted):
    ids, x, ys, w, dxs, dy = inputs(T, topk, E, H, dtype, T + H, drop)
    rows, slots, offsets = sort_ref(ids, E)
    kept = int(offsets[E])
    eps = torch.finfo(dtype).eps if dtype != torch.float32 else 0.0
    order = api.moe_sort(ids.to(dev()), E)
    xg, yg, wg = (t.to(dev()).requires_grad_() for t in (x, ys, w))
    xs = api.moe_permute(xg, order)
    y = api.moe_unpermute(yg, order, wg if weighted else None)
    asked = (xg, yg, wg) if weighted else (xg, yg)
    grads = torch.autograd.grad((xs, y), asked, (dxs.to(dev()), dy.to(dev())))

    token = slots // topk
    want = x[token].clone()
    want[kept:] = 0
    assert torch.equal(xs.cpu(), want)
    here = (rows < kept).double()
    ww = (w.double() if weighted else torch.ones(T, topk, dtype=torch.float64)) * here
    by_slot = ys.double()[rows.reshape(-1)].view(T, topk, H)
    close(y, (ww[:, :, None] * by_slot).sum(1), eps, topk, (ww[:, :, None] * by_slot.abs()).sum(1))
    back = dxs.double()[rows.reshape(-1)].view(T, topk, H) * here[:, :, None]
    close(grads[0], back.sum(1), eps, topk, back.abs().sum(1))
    wr = ww.reshape(-1)[slots][:, None]
    close(grads[1], wr * dy.double()[token], eps, 1, (wr * dy.double()[token]).abs())
    if weighted:
        prod = by_slot * dy.double()[:, None, :] * here[:, :, None]
        close(grads[2], prod.sum(2), 0.0, H, prod.abs().sum(2))
        assert bool((grads[2].cpu()[here == 0] == 0).all())


def test_rows_without_an_expert_are_not_read():
    """NaN in them reaches no output and no gradient."""
    ids, x, ys, w, _, dy = inputs(40, 4, 6, 96, torch.bfloat16, 2, 0.5)
    order = api.moe_sort(ids.to(dev()), 6)
    kept = int(order.offsets[6])
    ys[kept:] = float("nan")
    yg, wg = ys.to(dev()).requires_grad_(), w.to(dev()).requires_grad_()
    y = api.moe_unpermute(yg, order, wg)
    grads = torch.autograd.grad(y, (yg, wg), dy.to(dev()))
    for t in (y, *grads):
        assert bool(torch.isfinite(t).all())
    assert bool((grads[0][kept:] == 0).all())
    none = api.moe_sort(torch.full((7, 2), -1, device=dev()), 6)
    assert bool((api.moe_unpermute(torch.full((14, 8), float("nan"), device=dev()), none) == 0).all())


def test_differences():
    """Gradients against differences of the forward pass, fp32."""
    T, topk, E, H = 6, 3, 5, 9
    ids, x, ys, w, dxs, dy = inputs(T, topk, E, H, torch.float32, 11, 0.3)
    order = api.moe_sort(ids.to(dev()), E)
    f = lambda x, ys, w: float((api.moe_permute(x, order) * dxs.to(dev())).double().sum() +
                               (api.moe_unpermute(ys, order, w) * dy.to(dev())).double().sum())
    base = [t.to(dev()) for t in (x, ys, w)]
    leaves = [t.clone().requires_grad_() for t in base]
    xs, y = api.moe_permute(leaves[0], order), api.moe_unpermute(leaves[1], order, leaves[2])
    grads = torch.autograd.grad((xs, y), leaves, (dxs.to(dev()), dy.to(dev())))
    for k, g in enumerate(grads):
        for i in range(0, g.numel(), 5):
            lo, hi = [t.clone() for t in base], [t.clone() for t in base]
            lo[k].view(-1)[i] -= 0.5
            hi[k].view(-1)[i] += 0.5
            # linear in each operand: the difference over one is the gradient, up to fp32 sums of
            # a few hundred terms of order one
            assert abs(f(*hi) - f(*lo) - float(g.view(-1)[i])) < 1e-3


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides(dtype):
    """Rows of wider matrices at odd offsets, and expanded gradients."""
    T, topk, E, H = 70, 2, 5, 131
    ids, x, ys, w, _, _ = inputs(T, topk, E, H + 9, dtype, 4, 0.2)
    order = api.moe_sort(ids.to(dev()), E)
    xw, yw = x.to(dev()), ys.to(dev())
    for lo in (0, 3, 8):
        xv, yv = xw[:, lo:lo + H], yw[:, lo:lo + H]
        assert torch.equal(api.moe_permute(xv, order), api.moe_permute(xv.contiguous(), order))
        assert torch.equal(api.moe_unpermute(yv, order, w.to(dev())), api.moe_unpermute(yv.contiguous(), order, w.to(dev())))
    leaf, wl = yw[:, :H].detach().clone().requires_grad_(), w.to(dev()).requires_grad_()
    api.moe_unpermute(leaf, order, wl).sum().backward()
    ones = torch.ones(T, H, dtype=dtype, device=dev())
    leaf2, wl2 = leaf.detach().clone().requires_grad_(), wl.detach().clone().requires_grad_()
    api.moe_unpermute(leaf2, order, wl2).backward(ones)
    assert torch.equal(leaf.grad, leaf2.grad) and torch.equal(wl.grad, wl2.grad)
    shared = torch.randn(1, H, device=dev()).to(dtype).requires_grad_()   # one row for all tokens
    api.moe_permute(shared.expand(T, H), order).sum().backward()
    kept = int(order.offsets[E])
    assert float((shared.grad.double() - kept).abs().max()) <= kept * torch.finfo(dtype).eps * 4


def test_empty():
    order = api.moe_sort(torch.empty(0, 2, dtype=torch.int64, device=dev()), 3)
    x = torch.empty(0, 8, device=dev(), requires_grad=True)
    xs = api.moe_permute(x, order)
    y = api.moe_unpermute(xs, order, torch.empty(0, 2, device=dev()))
    assert xs.shape == (0, 8) and y.shape == (0, 8)
    y.sum().backward()
    assert x.grad.shape == (0, 8)


def test_captured_training_step():
    """Sort, rows there and back and their gradients, captured, replayed on new ids."""
    T, topk, E, H = 3000, 4, 16, 200
    g = torch.Generator().manual_seed(1)
    ids = make_ids(T, topk, E, 1, 0.1).to(dev())
    x, w = torch.randn(T, H, generator=g).to(dev()), torch.rand(T, topk, generator=g).to(dev())

    def step():
        xl, wl = x.detach().requires_grad_(), w.detach().requires_grad_()
        order = api.moe_sort(ids, E)
        y = api.moe_unpermute(api.moe_permute(xl, order), order, wl)
        return (y.detach(),) + torch.autograd.grad(y, (xl, wl), x)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (2, 3, 4):
        ids.copy_(make_ids(T, topk, E, seed, 0.1))
        x.add_(1.0)
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_capture_with_a_live_eager_graph_is_refused():
    """An eager graph of the same leaf on the default stream, alive: refused, not the process's end."""
    ids = make_ids(20, 2, 4, 1).to(dev())
    order = api.moe_sort(ids, 4)
    x = torch.randn(20, 8, device=dev(), requires_grad=True)
    alive = api.moe_permute(x, order)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="captured"):
        with torch.cuda.graph(graph):
            api.moe_permute(x, order).sum().backward()
    torch.cuda.synchronize()
    assert alive.shape == (40, 8)


def test_no_second_derivatives():
    order = api.moe_sort(make_ids(5, 2, 3, 1).to(dev()), 3)
    x = torch.randn(5, 8, device=dev(), requires_grad=True)
    xs = api.moe_permute(x, order)
    g, = torch.autograd.grad(xs.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), x)
    y = api.moe_unpermute(api.moe_permute(x, order), order, torch.ones(5, 2, device=dev()))
    g, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), x)
