"""What the autograd form of the 128-block layer keeps, and for how long; two
streams at once; the step captured into a graph."""

import pytest
import torch

from mxfp8_block_scaled_amd import api
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

M, N, K = 512, 1024, 2048
PACKED_X = M * K * 33 // 32                      # E4M3 and scale bytes
PACKED_WT = N * K + (N // 128) * (K // 128) * 4  # transposed weight and its scales
SLACK = 4 * 512                                  # the allocator's rounding of four tensors


def leaves(seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).to(dev())
    w = (torch.randn(N, K, generator=g) * 0.02).to(torch.bfloat16).to(dev())
    b = torch.randn(N, generator=g).to(torch.bfloat16).to(dev())
    return [t.requires_grad_() for t in (x, w, b)]


def test_kept_memory_goes_with_the_backward_pass():
    x, w, b = leaves()
    dy = torch.ones(M, N, dtype=torch.bfloat16, device=dev())
    torch.autograd.grad(api.linear_b128(x, w, b), (x, w, b), dy)   # first-call allocations
    start = torch.cuda.memory_allocated()
    y = api.linear_b128(x, w, b)
    kept = torch.cuda.memory_allocated() - start - y.numel() * 2
    assert PACKED_X + PACKED_WT <= kept <= PACKED_X + PACKED_WT + SLACK
    torch.autograd.grad(y, (x, w, b), dy)
    # y and its graph live on, what was kept does not
    assert torch.cuda.memory_allocated() - start - y.numel() * 2 <= SLACK
    with pytest.raises(RuntimeError, match="second time"):
        torch.autograd.grad(y, (x, w, b), dy)


def test_nothing_is_kept_without_gradients():
    x, w, b = leaves()
    y0 = api.linear_b128(x, w, b)
    torch.cuda.synchronize()
    start = torch.cuda.memory_allocated()
    with torch.no_grad():
        y = api.linear_b128(x, w, b)
    assert not y.requires_grad and torch.cuda.memory_allocated() - start <= y.numel() * 2 + SLACK
    assert torch.equal(y, y0)


def test_recomputed_layer():
    """Under torch's activation checkpointing the kept bytes are made again."""
    from torch.utils.checkpoint import checkpoint
    x, w, b = leaves()
    dy = torch.randn(M, N, device=dev()).to(torch.bfloat16)
    want = torch.autograd.grad(api.linear_b128(x, w, b), (x, w, b), dy)
    y = checkpoint(api.linear_b128, x, w, b, use_reentrant=False)
    for g, h in zip(torch.autograd.grad(y, (x, w, b), dy), want):
        assert torch.equal(g, h)


def test_two_streams_at_once():
    """Steps of different data in flight on two streams share nothing."""
    sets = [leaves(s) for s in (1, 2)]
    dy = torch.randn(M, N, device=dev()).to(torch.bfloat16)
    want = [[y.detach().clone() for y in (o, *torch.autograd.grad(o, s, dy))]
            for s in sets for o in [api.linear_b128(*s)]]
    logits = [torch.randn(2000, 64, device=dev()) for _ in sets]
    loss = [api.moe_balance(l, 4, z_coef=1e-3)[0].clone() for l in logits]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got, got_loss = [[], []], [[], []]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                y = api.linear_b128(*sets[i])
                got[i].append([y, *torch.autograd.grad(y, sets[i], dy)])
                got_loss[i].append(api.moe_balance(logits[i], 4, z_coef=1e-3)[0])
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            for g, h in zip(run, want[i]):
                assert torch.equal(g, h)
        for l in got_loss[i]:
            assert torch.equal(l, loss[i])


def test_captured_step_replays():
    """Forward and gradients of the layer and of the balance loss, captured and
    replayed on new values between eager work."""
    x, w, b = leaves()
    l = torch.randn(700, 64, device=dev()).requires_grad_()
    dy = torch.randn(M, N, device=dev()).to(torch.bfloat16)

    def step():
        y = api.linear_b128(x, w, b)
        loss, counts = api.moe_balance_loss(l, 4, z_coef=1e-3)
        return [y.detach(), loss.detach(), counts, *torch.autograd.grad(y, (x, w, b), dy),
                *torch.autograd.grad(loss, l)]

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    torch.cuda.current_stream().wait_stream(st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in (3, 4, 5):
        with torch.no_grad():
            for t, n in zip((x, w, b), leaves(seed)):
                t.copy_(n)
            l.copy_(torch.randn(700, 64, device=dev()))
        g.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, step()):
            assert torch.equal(p, q)


def test_capture_beside_a_living_graph_is_refused():
    """The backward pass raises before it hands anything to torch's
    accumulators; the capture ends in order and everything goes on working."""
    x, w, b = leaves()
    dy = torch.randn(M, N, device=dev()).to(torch.bfloat16)
    alive = api.linear_b128(x, w, b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="alive on another stream"):
        with torch.cuda.graph(g):
            y = api.linear_b128(x, w, b)
            torch.autograd.grad(y, (x, w, b), dy)
    torch.cuda.synchronize()
    want = torch.autograd.grad(alive, (x, w, b), dy)
    again = torch.autograd.grad(api.linear_b128(x, w, b), (x, w, b), dy)
    for p, q in zip(again, want):
        assert torch.equal(p, q)


def test_second_derivative_is_an_error():
    x, w, b = leaves()
    dy = torch.ones(M, N, dtype=torch.bfloat16, device=dev())
    plain = torch.autograd.grad(api.linear_b128(x, w, b), (x, w, b), dy)
    dx, dw, db = torch.autograd.grad(api.linear_b128(x, w, b), (x, w, b), dy.requires_grad_(), create_graph=True)
    assert all(torch.equal(g, h) for g, h in zip((dx, dw, db), plain))
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dw.float().sum().backward()
