"""The router's balance and z loss, expert counts and gradient against a
64-bit form; masks that leave rows or everything out; ties; non-finite
logits; agreement with the routed layer's own selection."""

import numpy as np
import pytest
import torch

from mxfp8_block_scaled_amd import api
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


def reference(logits, k, valid, coef, z_coef, counts=None, used=None):
    """(loss, counts, n, gradient) in 64 bits."""
    x = logits.detach().cpu().double().numpy()
    T, E = x.shape
    live = ~(x == -np.inf).all(1)
    if valid is not None:
        live &= valid.cpu().numpy().astype(bool)
    x = x[live]
    n = int(live.sum()) if used is None else used
    with np.errstate(invalid="ignore"):
        m = x.max(1, keepdims=True) if len(x) else x[:, :1]
        e = np.exp(x - m)
        p = e / e.sum(1, keepdims=True)
        lse = (m + np.log(e.sum(1, keepdims=True)))
    own = np.zeros(E, dtype=np.int64)
    for r in np.where(np.isnan(x), -np.inf, x):
        own[np.lexsort((np.arange(E), -r))[:k]] += 1
    c = own if counts is None else counts
    d = max(n, 1)
    a, b = coef * E / (k * float(d) ** 2), z_coef / d
    loss = a * (c * p.sum(0)).sum() + b * (lse ** 2).sum()
    grad = np.zeros((T, E))
    grad[live] = a * p * (c - (p * c).sum(1, keepdims=True)) + 2 * b * lse * p
    scale = np.zeros((T, 1))
    scale[live] = a * (c.max(initial=0) + 1) + 2 * abs(b) * np.abs(lse)
    return loss, own, n, grad, scale


def check(logits, k, valid=None, coef=1e-2, z_coef=1e-3):
    loss, counts, used = api.moe_balance(logits, k, valid=valid, coef=coef, z_coef=z_coef)
    grad = api.moe_balance_backward(logits, k, counts, used, valid=valid, coef=coef, z_coef=z_coef)
    want, wc, n, wg, scale = reference(logits, k, valid, coef, z_coef)
    assert counts.dtype == torch.int32 and np.array_equal(counts.cpu().numpy(), wc)
    assert int(used) == n
    # exp, log and the divisions are good to a few 2^-24 of their values for
    # exponents below 2^5 in magnitude (2^-19 allowed); sums of at most
    # 2^8 + 2^8 terms per lane and workgroup add 2^-24 each (2^-15 allowed)
    assert abs(float(loss) - want) <= 2.0 ** -15 * (abs(want) + 1e-30), (float(loss), want)
    err = np.abs(grad.double().cpu().numpy() - wg)
    bound = 2.0 ** -16 * scale + 1e-38
    if logits.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * np.abs(wg)
    assert grad.dtype == logits.dtype and (err <= bound).all(), float((err / bound).max())
    return loss, counts, used, grad


def make(T, E, seed, dtype=torch.float32, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * spread + torch.randn(E, generator=g)).to(dtype).to(dev())


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (16, 8, 8), (63, 16, 1), (64, 17, 16), (65, 60, 4),
                                   (300, 64, 6), (1000, 128, 8), (77, 160, 3), (5000, 256, 8), (17000, 40, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sizes(T, E, k, dtype):
    check(make(T, E, T + E, dtype), k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["bool", "uint8"])
def test_masked_tokens(dtype, kind):
    logits = make(500, 32, 1, dtype)
    valid = torch.rand(500, generator=torch.Generator().manual_seed(2)) < 0.6
    logits[~valid.to(dev())] = float("nan")          # what lies in padding does not matter
    valid = valid.to(dev()) if kind == "bool" else (valid * 3).to(torch.uint8).to(dev())
    _, counts, used, grad = check(logits, 4, valid)
    assert int(counts.sum()) == 4 * int(used)
    assert not grad[valid == 0].any()


def test_nothing_counted():
    logits = make(70, 24, 3)
    loss, counts, used, grad = check(logits, 2, torch.zeros(70, dtype=torch.bool, device=dev()))
    assert float(loss) == 0 and not counts.any() and int(used) == 0 and not grad.any()
    loss, counts, used, grad = check(torch.full((9, 24), -float("inf"), device=dev()), 2)
    assert float(loss) == 0 and not counts.any() and int(used) == 0 and not grad.any()
    loss, counts, used, grad = check(torch.empty(0, 24, device=dev()), 2)
    assert float(loss) == 0 and not counts.any() and grad.shape == (0, 24)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_experts_and_lowest_values(dtype):
    logits = make(130, 48, 4, dtype)
    logits[:, 5:20] = -float("inf")
    logits[3, :] = -float("inf")                     # a row with nothing left
    logits[4, 1:] = -float("inf")                    # fewer finite logits than k
    logits[5, :] = torch.finfo(dtype).min            # a mask of the type's lowest value
    logits[6, 1:] = torch.finfo(dtype).min
    check(logits, 4, z_coef=0.0)
    check(logits[torch.arange(130, device=dev()) % 7 < 5][10:], 4)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_take_the_lower_expert(dtype):
    g = torch.Generator().manual_seed(5)
    logits = torch.randint(0, 3, (400, 64), generator=g).to(dtype).to(dev())
    logits[::2] *= -1                                # zeros of both signs
    check(logits, 6)
    check(torch.zeros(10, 100, dtype=dtype, device=dev()), 3)


def test_non_finite_logits():
    logits = make(100, 32, 6)
    logits[40, 3] = float("nan")
    logits[41, 4] = float("inf")
    loss, counts, used = api.moe_balance(logits, 2)
    grad = api.moe_balance_backward(logits, 2, counts, used)
    assert loss.isnan() and int(used) == 100 and int(counts.sum()) == 200
    bad = torch.zeros(100, dtype=torch.bool, device=dev())
    bad[40:42] = True
    assert torch.equal(grad.isnan().any(1), bad)


def test_counts_are_the_routed_layers():
    T, H, E, k, I = 96, 256, 16, 4, 256
    g = torch.Generator().manual_seed(7)
    logits = torch.randint(-4, 5, (T, E), generator=g).float().to(dev())
    w = [torch.randint(0, 120, s, generator=g, dtype=torch.uint8).to(dev()) for s in ((E, 2 * I, H), (E, H, I))]
    s = [torch.full((*t.shape[:2], t.shape[2] // 32), 110, dtype=torch.uint8, device=dev()) for t in w]
    mw = api.moe_prepare_weights(w[0], s[0], w[1], s[1])
    ids = torch.empty(T * k, dtype=torch.int32, device=dev())
    act = torch.empty(T * k, I, dtype=torch.bfloat16, device=dev())
    q, sc = torch.empty(T * k, I, dtype=torch.uint8, device=dev()), torch.empty(T * k, I // 32, dtype=torch.uint8, device=dev())
    wts = torch.empty(T * k, device=dev())
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(dev())
    api.moe_debug_capture(act, q, sc, ids, wts)
    try:
        api.moe_grouped(x, logits, mw, k)
        torch.cuda.synchronize()
    finally:
        api.moe_debug_capture()
    _, counts, _ = api.moe_balance(logits, k)
    assert torch.equal(counts.long(), torch.bincount(ids.long(), minlength=E))


def test_autograd_and_upstream_gradient():
    logits = make(333, 40, 8).requires_grad_()
    valid = torch.arange(333, device=dev()) % 5 != 0
    loss, counts = api.moe_balance_loss(logits, 4, valid, coef=0.1, z_coef=0.01)
    assert not counts.requires_grad
    (loss * 3.5).backward()
    want = reference(logits, 4, valid, 0.1, 0.01)
    assert np.array_equal(counts.cpu().numpy(), want[1])
    err = np.abs(logits.grad.double().cpu().numpy() - 3.5 * want[3])
    assert (err <= 3.5 * (2.0 ** -16 * want[4] + 1e-38)).all()


def test_gradient_against_differences():
    """Central differences of the 64-bit loss with the counts held."""
    logits = make(12, 6, 9)
    loss, counts, used = api.moe_balance(logits, 2, coef=1.0, z_coef=0.1)
    grad = api.moe_balance_backward(logits, 2, counts, used, coef=1.0, z_coef=0.1).double().cpu().numpy()
    c, h = counts.cpu().numpy(), 2.0 ** -10
    for t in range(12):
        for e in range(6):
            up, dn = logits.cpu().double(), logits.cpu().double()
            up[t, e] += h
            dn[t, e] -= h
            slope = (reference(up, 2, None, 1.0, 0.1, c, 12)[0] - reference(dn, 2, None, 1.0, 0.1, c, 12)[0]) / (2 * h)
            # h^2 / 6 times a third derivative below 10, and the fp32 gradient
            assert abs(slope - grad[t, e]) <= h * h * 2 + 1e-5 * max(1.0, abs(slope))


def test_counts_summed_over_ranks():
    """Two halves' counts and tokens added give the whole batch's gradient."""
    logits = make(400, 32, 10)
    _, c, n = api.moe_balance(logits, 4)
    parts = [api.moe_balance(h, 4) for h in logits.chunk(2)]
    cs, ns = parts[0][1] + parts[1][1], parts[0][2] + parts[1][2]
    assert torch.equal(cs, c) and torch.equal(ns, n)
    whole = api.moe_balance_backward(logits, 4, c, n)
    halves = [api.moe_balance_backward(h, 4, cs, ns) for h in logits.chunk(2)]
    assert torch.equal(whole, torch.cat(halves))


def test_strided_logits():
    wide = make(90, 100, 11)
    view = wide[:, 30:62]
    a, b = api.moe_balance(view, 4), api.moe_balance(view.contiguous(), 4)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    ga = api.moe_balance_backward(view, 4, *a[1:])
    assert torch.equal(ga, api.moe_balance_backward(view.contiguous(), 4, *b[1:]))
    row = wide[:1, :32].expand(50, 32)
    check(row, 4)


@pytest.mark.parametrize("T", [40, 20000])
def test_graph_replays(T):
    logits = make(T, 64, 0, torch.bfloat16)

    def step():
        loss, counts, used = api.moe_balance(logits, 4, z_coef=1e-3)
        return loss, counts, used, api.moe_balance_backward(logits, 4, counts, used, z_coef=1e-3)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in range(4):
        logits.copy_(make(T, 64, seed, torch.bfloat16))
        want = step()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
