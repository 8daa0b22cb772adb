"""Which captured backward passes are refused, on the CPU with streams as plain
values: those that would make the legacy default stream (0) wait for the
capture, or may.  A capture takes in any other stream.  (Nothing is captured
here; tests/test_gpu_capture_streams.py captures.)"""

import pytest
import torch

from mxfp8_block_scaled_amd import api


@pytest.fixture
def stream(monkeypatch):
    """Sets the current stream."""
    now = [0]
    monkeypatch.setattr(api, "_stream", lambda device=None: now[0])

    def use(s):
        now[0] = s
    return use


def leaves(n=2):
    return [torch.ones(3, requires_grad=True) for _ in range(n)]


def call(x, w, s):
    """An operator of this library on stream s, as far as its graph goes."""
    api._mark_leaves_before((x, w), s)
    out = x * w
    api._mark_leaves(out, s)
    return out


def refused(out, s):
    try:
        api._check_capture(out.grad_fn, s, capturing=True)
    except RuntimeError:
        return True
    return False


def test_warm_up_on_a_side_stream_stays_alive(stream):
    x, w = leaves()
    stream(5)
    warm = call(x, w, 5)
    warm.sum().backward()
    stream(7)
    assert not refused(call(x, w, 7), 7)
    assert warm.grad_fn is not None


def test_default_stream_graph_stays_alive(stream):
    x, w = leaves()
    old = call(x, w, 0)
    stream(7)
    assert refused(call(x, w, 7), 7)
    del old
    assert not refused(call(x, w, 7), 7)


@pytest.mark.parametrize("alive", [True, False])
def test_accumulator_of_another_operator(stream, alive):
    """Made where this library did not see it, so its stream is not known: not
    at the capture, nor by a warm-up that only asks for gradients."""
    x, w = leaves()
    other = w * 2.0
    if not alive:
        del other
    assert refused(call(x, w, 7), 7) == alive
    stream(5)
    warm = call(x, w, 5)
    torch.autograd.grad(warm.sum(), (x, w))
    assert refused(call(x, w, 7), 7) == alive


@pytest.mark.parametrize("home", [0, 5])
def test_a_backward_pass_shows_the_stream(stream, home):
    """Accumulators held by something else for good, as a data-parallel wrapper
    does.  torch runs an accumulator on its own stream."""
    x, w = leaves()
    held = [torch.autograd.graph.get_gradient_edge(t) for t in (x, w)]
    stream(5)
    for _ in range(2):
        warm = call(x, w, 5)
        stream(home)
        warm.sum().backward()
        stream(5)
    stream(7)
    assert refused(call(x, w, 7), 7) == (home == 0)
    assert len(held) == 2


def test_the_captured_stream_itself(stream):
    x, w = leaves()
    stream(7)
    old = call(x, w, 7)
    assert not refused(call(x, w, 7), 7)
    assert not refused(old, 7)


def test_operands_without_gradients_and_computed_ones(stream):
    x = torch.ones(3)
    w, = leaves(1)
    stream(7)
    api._mark_leaves_before((x, w * 1.0, None), 7)
    assert not refused(call(x, w, 7), 7)
    assert not refused(call(w * 1.0, w * 2.0, 7), 7)
