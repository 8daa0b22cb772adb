"""Training steps captured after a warm-up on a side stream, with what the
warm-up made still alive; and those that have to be refused.  Replays on new
values against the same step run at once on leaves of its own."""

import gc

import pytest
import torch

from mxfp8_block_scaled_amd import api
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

M, N, K, T, E = 200, 144, 272, 500, 32
REFUSED = "alive on another stream"


@pytest.fixture(autouse=True)
def nothing_left_behind():
    """Graphs and the refusals' tracebacks hold tensors in cycles."""
    yield
    torch.cuda.synchronize()
    gc.collect()


def leaves(seed):
    g = torch.Generator().manual_seed(seed)
    bf16 = [torch.randn(s, generator=g).to(torch.bfloat16).to(dev()) for s in ((M, K), (N, K), (N,))]
    return [t.requires_grad_() for t in bf16 + [torch.randn(T, E, generator=g).to(dev())]]


DY = torch.randn(M, N, generator=torch.Generator().manual_seed(99)).to(torch.bfloat16)


def step(ts, dy):
    """Forward, backward() into the leaves; the outputs with their graph."""
    y = api.linear_b128(*ts[:3])
    loss, counts = api.moe_balance_loss(ts[3], 4, z_coef=1e-3)
    torch.autograd.backward([y, loss], [dy, None])
    return y, loss, counts


def clear(ts):
    for t in ts:
        t.grad = None


def side_stream(work):
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        out = work()
    torch.cuda.current_stream().wait_stream(st)
    return out


def check_replays(g, ts, got, dy):
    for seed in (3, 4, 5):
        fresh = leaves(seed)
        with torch.no_grad():
            for t, n in zip(ts, fresh):
                t.copy_(n)
        g.replay()
        torch.cuda.synchronize()
        want = step(fresh, dy)
        torch.cuda.synchronize()
        for p, q in zip(got, want):
            assert torch.equal(p, q)
        for t, n in zip(ts, fresh):
            assert torch.equal(t.grad, n.grad)


def test_warm_up_outputs_stay_alive():
    ts, dy = leaves(0), DY.to(dev())

    def warm():
        for _ in range(3):
            clear(ts)
            out = step(ts, dy)
        return out

    alive = side_stream(warm)
    clear(ts)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(ts, dy)
    check_replays(g, ts, got, dy)
    assert alive[0].grad_fn is not None and alive[1].grad_fn is not None


def test_accumulators_held_from_the_side_stream():
    """As a data-parallel wrapper that was made there holds them."""
    ts, dy = leaves(1), DY.to(dev())

    def warm():
        held = [torch.autograd.graph.get_gradient_edge(t) for t in ts]
        for _ in range(2):
            clear(ts)
            step(ts, dy)
        return held

    held = side_stream(warm)
    clear(ts)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(ts, dy)
    check_replays(g, ts, got, dy)
    assert len(held) == len(ts)


def test_graphed_callable():
    """torch.cuda.make_graphed_callables, which warms up on a side stream and
    keeps the last outputs."""
    class Layer(torch.nn.Module):
        def __init__(self, w, b):
            super().__init__()
            self.w, self.b = torch.nn.Parameter(w), torch.nn.Parameter(b)

        def forward(self, x):
            return api.linear_b128(x, self.w, self.b)

    x, w, b, _ = (t.detach() for t in leaves(6))
    dy = DY.to(dev())
    graphed = torch.cuda.make_graphed_callables(Layer(w.clone(), b.clone()), (x.clone().requires_grad_(),))
    for seed in (7, 8, 9):
        xs = leaves(seed)[0], leaves(seed)[0]
        plain = Layer(w.clone(), b.clone())
        for p in graphed.parameters():
            p.grad = None
        y, want = graphed(xs[0]), plain(xs[1])
        y.backward(dy)
        want.backward(dy)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(xs[0].grad, xs[1].grad)
        for p, q in zip(graphed.parameters(), plain.parameters()):
            assert torch.equal(p.grad, q.grad)


@pytest.mark.parametrize("warmed", [False, True])
def test_accumulators_held_from_the_default_stream(warmed):
    """Not seen here before the capture, or seen on a side stream only."""
    ts, dy = leaves(2), DY.to(dev())
    held = [torch.autograd.graph.get_gradient_edge(t) for t in ts]
    if warmed:
        side_stream(lambda: step(ts, dy) and None)
        homes = [h.node.metadata["mxfp8_stream"] for h in held]
        assert homes == [0] * len(ts)
        clear(ts)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match=REFUSED):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            y = api.linear_b128(*ts[:3])
            torch.autograd.grad(y, ts[:3], dy)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match=REFUSED):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            loss, _ = api.moe_balance_loss(ts[3], 4)
            torch.autograd.grad(loss, ts[3])
    torch.cuda.synchronize()
    clear(ts)
    step(ts, dy)
    fresh = leaves(2)
    step(fresh, dy)
    for t, n in zip(ts, fresh):
        assert torch.equal(t.grad, n.grad)
