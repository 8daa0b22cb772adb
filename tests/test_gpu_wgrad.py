"""Weight and bias gradients from 8-bit activation checkpoints, and the
128-block layer's training step, against 64-bit forms."""

import numpy as np
import pytest
import torch

from mxfp8_block_scaled_amd import api
from tests import b128_ref as ref
from tests.gpu_util import dev
from tests.test_gpu_b128 import f64, randn, spiky

pytestmark = pytest.mark.gpu


def keep(x, form):
    return (api.quantize_act_packed if form == "mx" else api.quantize_act_packed_b128)(x.to(dev()))


def check_dw(dw, db, dy, X, base=None, base_b=None):
    """Products are exact and every fp32 addition rounds by at most 2^-24 of
    the sum of magnitudes: M + 32 of them (tokens, splits, the accumulation)
    are allowed 2^-23 each; bf16 outputs add one rounding."""
    d = f64(dy)
    M = d.shape[0]
    for got, want, mag in ((dw, d.T @ X, np.abs(d).T @ np.abs(X)),
                           (db, d.sum(0), np.abs(d).sum(0))):
        if got is None:
            continue
        b = base if got is dw else base_b
        if b is not None:
            want, mag = want + f64(b), mag + np.abs(f64(b))
        bound = (M + 32) * 2.0 ** -23 * mag + 2.0 ** -140
        if got.dtype == torch.bfloat16:
            bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
        err = np.abs(f64(got) - want)
        assert np.isfinite(f64(got)).all()
        assert (err <= bound).all(), (float((err / bound).max()), np.argwhere(err > bound)[:4])


SIZES = [(1, 8, 16, "b128"), (2, 16, 256, "mx"), (31, 136, 144, "b128"), (64, 128, 128, "b128"), (65, 120, 272, "b128"),
         (127, 256, 256, "mx"), (128, 136, 400, "b128"), (129, 512, 512, "mx"), (300, 520, 1040, "b128"),
         (1000, 264, 2064, "b128"), (1030, 1024, 1024, "mx"), (4100, 128, 128, "b128"), (2048, 2304, 2304, "mx")]


@pytest.mark.parametrize("M,N,K,form", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wgrad(M, N, K, form, dtype):
    x, dy = spiky(M, K, M + K), randn((M, N), N, 1e-3)
    pa = keep(x, form)
    X = f64(pa.dequantize())
    dw, db = api.linear_wgrad(dy.to(dev()), pa, dtype=dtype, bias_grad=True)
    assert dw.dtype == dtype and dw.shape == (N, K) and db.dtype == torch.float32
    check_dw(dw, db, dy, X)
    half = torch.empty(N, dtype=torch.bfloat16, device=dev())
    assert api.linear_wgrad(dy.to(dev()), pa, dtype=dtype, bias_grad=True, out_bias=half)[1] is half
    assert torch.equal(half, db.to(torch.bfloat16))
    assert torch.equal(dw, api.linear_wgrad(dy.to(dev()), pa, dtype=dtype))


@pytest.mark.parametrize("M,N,K,form", [(65, 136, 272, "b128"), (2000, 264, 512, "mx")])
def test_wgrad_accumulates(M, N, K, form):
    x, dy = spiky(M, K, 1), randn((M, N), 2)
    pa = keep(x, form)
    base, base_b = torch.randn(N, K) * 10, torch.randn(N) * 10
    out, out_b = base.to(dev()), base_b.to(dev())
    dw, db = api.linear_wgrad(dy.to(dev()), pa, bias_grad=True, out=out, out_bias=out_b, accumulate=True)
    assert dw is out and db is out_b
    check_dw(dw, db, dy, f64(pa.dequantize()), base, base_b)


def test_wgrad_of_no_tokens():
    pa = api.quantize_act_packed_b128(torch.empty(0, 64, dtype=torch.bfloat16, device=dev()))
    dy = torch.empty(0, 24, dtype=torch.bfloat16, device=dev())
    dw, db = api.linear_wgrad(dy, pa, bias_grad=True)
    assert not dw.any() and not db.any() and dw.shape == (24, 64)
    out, ob = torch.ones(24, 64, device=dev()), torch.ones(24, device=dev())
    api.linear_wgrad(dy, pa, bias_grad=True, out=out, out_bias=ob, accumulate=True)
    assert (out == 1).all() and (ob == 1).all()


def test_wgrad_one_token_places_every_element():
    """M = 1: each output is one exact product."""
    x, dy = spiky(1, 528, 3), randn((1, 264), 4)
    pa = keep(x, "b128")
    dw, db = api.linear_wgrad(dy.to(dev()), pa, bias_grad=True)
    assert np.array_equal(f64(dw), np.outer(f64(dy)[0], f64(pa.dequantize())[0]).astype(np.float32).astype(float))
    assert np.array_equal(f64(db), f64(dy)[0])


def test_wgrad_one_hot_tokens():
    """dY picks one token per output row: rows of the checkpoint, exactly, from
    every position of a step, a 128-row group and a split run."""
    M, N, K = 700, 704, 400
    x = spiky(M, K, 5)
    pa = keep(x, "b128")
    perm = torch.randperm(M, generator=torch.Generator().manual_seed(2))
    dy = torch.zeros(M, N, dtype=torch.bfloat16)
    dy[perm, torch.arange(M)] = 1.0
    dw = api.linear_wgrad(dy.to(dev()), pa)
    want = np.zeros((N, K))
    want[:M] = f64(pa.dequantize())[perm.numpy()]
    assert np.array_equal(f64(dw), want)


def test_wgrad_strides_and_surroundings():
    M, N, K = 190, 136, 272
    x = spiky(M, K, 6)
    pa = keep(x, "b128")
    X = f64(pa.dequantize())
    wide = randn((M, N + 64), 7).to(dev())
    wide[:, :32] = float("nan")                      # neighbours of the view
    wide[:, 32 + N:] = float("nan")
    dy = wide[:, 32:32 + N]
    out = torch.full((N + 2, K + 16), 5.0, device=dev())
    dw = api.linear_wgrad(dy, pa, out=out[1:N + 1, :K])
    check_dw(dw, None, dy.cpu(), X)
    edge = out.clone()
    edge[1:N + 1, :K] = 5.0
    assert (edge == 5.0).all()
    ones = torch.ones((), dtype=torch.bfloat16, device=dev()).expand(M, N)   # the gradient of a sum
    check_dw(*api.linear_wgrad(ones, pa, bias_grad=True), ones.cpu(), X)
    tr = randn((N, M), 8).to(dev()).t()
    check_dw(api.linear_wgrad(tr, pa), None, tr.cpu(), X)


def test_wgrad_non_finite():
    """A NaN in dY reaches its column's gradients alone, a NaN block of the
    checkpoint its 128 input channels alone."""
    M, N, K = 130, 136, 400
    x, dy = randn((M, K), 1), randn((M, N), 2)
    x[100, 200] = float("nan")
    dy[7, 33] = float("inf")
    dw, db = api.linear_wgrad(dy.to(dev()), keep(x, "b128"), bias_grad=True)
    bad = torch.zeros(N, K, dtype=torch.bool)
    bad[:, 128:256] = True
    bad[33, :] = True
    assert torch.equal(~dw.cpu().isfinite(), bad)
    assert db.cpu().isfinite().sum() == N - 1


def test_wgrad_graph_replays():
    M, N, K = 1500, 264, 512
    dy, pa = randn((M, N), 1).to(dev()), keep(spiky(M, K, 1), "mx")
    api.linear_wgrad(dy, pa, bias_grad=True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dw, db = api.linear_wgrad(dy, pa, bias_grad=True)
    for seed in range(4):
        dy.copy_(randn((M, N), seed))
        want = api.linear_wgrad(dy, pa, bias_grad=True)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dw, want[0]) and torch.equal(db, want[1])


# ---------------------------------------------------------------- the layer under training

def train_reference(x, w, b, dy):
    _, _, A = ref.quantize(f64(x))
    _, _, W = ref.quantize(f64(w), rows=128)
    _, _, D = ref.quantize(f64(dy))
    return A, W, D


def check_close(got, want, bound):
    err = np.abs(f64(got) - want)
    lim = 2.0 ** -8 * np.abs(want) + bound
    assert (err <= lim).all(), float((err / lim).max())


@pytest.mark.parametrize("shape,N,K", [((5,), 16, 32), ((2, 33), 144, 272), ((300,), 528, 400), ((1100,), 1024, 512)])
def test_linear_b128_step(shape, N, K):
    x, w, b = spiky(int(np.prod(shape)), K, 1).view(*shape, K), spiky(N, K, 2), randn((N,), 3)
    dy = randn((*shape, N), 4, 1e-2)
    leaves = [t.to(dev()).requires_grad_() for t in (x, w, b)]
    y = api.linear_b128(*leaves)
    dx, dw, db = torch.autograd.grad(y, leaves, dy.to(dev()))
    assert y.shape == (*shape, N) and dx.shape == x.shape and dw.shape == w.shape
    x2, d2 = x.view(-1, K), dy.view(-1, N)
    A, W, D = train_reference(x2, w, b, d2)
    check_close(y.view(-1, N), A @ W.T + f64(b), ref.gemm_bound(A, W))
    check_close(dx.view(-1, K), D @ W, ref.gemm_bound(D, W.T))
    check_dw(dw, None, d2, A)
    want = f64(d2).sum(0)
    check_close(db, want, (d2.shape[0] + 32) * 2.0 ** -23 * np.abs(f64(d2)).sum(0) * (1 + 2.0 ** -8))


def test_linear_b128_gradient_against_differences():
    """Operands whose quantization is exact: dw and dx against differences of
    the layer's sums.  The differences are taken of the exact sums, not of the
    layer's bf16 outputs: 48 products of up to 8 * 15 need twelve bits and bf16
    holds eight.  dw and dx are integers below 2^11 rounded once to bf16."""
    M, N, K = 40, 32, 48
    g = torch.Generator().manual_seed(0)
    w = torch.randint(-8, 9, (N, K), generator=g).to(torch.bfloat16)
    w[0, 0] = 16.0    # fixes the block's scale
    x = torch.randint(-8, 9, (M, K), generator=g).to(torch.bfloat16)
    x[:, 0] = 15.0
    dy = torch.randint(-3, 4, (M, N), generator=g).to(torch.bfloat16)
    lw = w.to(dev()).requires_grad_()
    lx = x.to(dev()).requires_grad_()
    y = api.linear_b128(lx, lw)
    dx, dw = torch.autograd.grad(y, (lx, lw), dy.to(dev()))

    def loss(xx, ww):
        A, W, _ = train_reference(xx, ww, None, dy)
        assert np.array_equal(A, f64(xx)) and np.array_equal(W, f64(ww))
        return ((A @ W.T) * f64(dy)).sum()

    def same(slope, got):
        return abs(slope - float(got)) <= 2.0 ** -8 * abs(slope)

    for n, k in ((1, 1), (5, 20), (31, 47)):
        up, dn = w.clone(), w.clone()
        up[n, k], dn[n, k] = 4.0, 2.0
        assert same((loss(x, up) - loss(x, dn)) / 2.0, dw[n, k])
    for m, k in ((1, 1), (39, 47)):
        up, dn = x.clone(), x.clone()
        up[m, k], dn[m, k] = 4.0, 2.0
        assert same((loss(up, w) - loss(dn, w)) / 2.0, dx[m, k])


def test_linear_b128_partial_gradients_and_none():
    x, w = spiky(20, 64, 1).to(dev()), spiky(32, 64, 2).to(dev())
    y0 = api.linear_b128(x, w)
    assert not y0.requires_grad
    lw = w.clone().requires_grad_()
    y = api.linear_b128(x, lw)
    y.float().sum().backward()
    ones = torch.ones(20, 32, dtype=torch.bfloat16)
    check_dw(lw.grad, None, ones, f64(api.quantize_act_packed_b128(x).dequantize()))
    lx = x.clone().requires_grad_()
    api.linear_b128(lx, w).float().sum().backward()
    full = [x.clone().requires_grad_(), w.clone().requires_grad_()]
    api.linear_b128(*full).float().sum().backward()
    assert torch.equal(lx.grad, full[0].grad) and torch.equal(lw.grad, full[1].grad)


def test_mx_layer_weight_gradient():
    """The MXFP8 layer's own quantized activations serve its gradient."""
    x, w, dy = spiky(200, 512, 1), randn((256, 512), 2, 0.02), randn((200, 256), 3)
    wq, ws = api.quantize_act(w.to(dev()))
    pw = api.prepare_weight(wq, ws)
    pa = api.quantize_act_packed(x.to(dev()))
    y = api.gemm_packed(pa, pw)
    assert y.shape == (200, 256)
    check_dw(api.linear_wgrad(dy.to(dev()), pa), None, dy, f64(pa.dequantize()))


@pytest.mark.parametrize("tile", [128, 256])
@pytest.mark.parametrize("M,N,K,form", [(1, 8, 16, "b128"), (64, 256, 256, "mx"), (65, 264, 272, "b128"), (200, 520, 512, "mx"),
                                        (1000, 248, 1040, "b128"), (5000, 768, 528, "b128"), (640, 2304, 2304, "mx")])
def test_wgrad_tile_forms(tile, M, N, K, form):
    """Each form on shapes of few and many tiles; runs that end inside a tile,
    at its border, and hold several; accumulation and bf16 through the join."""
    x, dy = spiky(M, K, M + K), randn((M, N), N, 1e-3)
    pa = keep(x, form)
    X = f64(pa.dequantize())
    base, base_b = torch.randn(N, K), torch.randn(N)
    prev = api.mxfp8_debug_force_wgrad(tile)
    try:
        dw, db = api.linear_wgrad(dy.to(dev()), pa, bias_grad=True)
        half = api.linear_wgrad(dy.to(dev()), pa, dtype=torch.bfloat16)
        acc = api.linear_wgrad(dy.to(dev()), pa, bias_grad=True, out=base.to(dev()), out_bias=base_b.to(dev()), accumulate=True)
        again = api.linear_wgrad(dy.to(dev()), pa)
        none = api.linear_wgrad(torch.empty(0, N, dtype=torch.bfloat16, device=dev()),
                                api.quantize_act_packed_b128(torch.empty(0, K, dtype=torch.bfloat16, device=dev())))
    finally:
        api.mxfp8_debug_force_wgrad(prev)
    check_dw(dw, db, dy, X)
    check_dw(half, None, dy, X)
    check_dw(*acc, dy, X, base, base_b)
    assert torch.equal(dw, again) and not none.any()


def test_linear_b128_of_no_tokens():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=dev(), requires_grad=True)
    w, b = spiky(32, 64, 1).to(dev()).requires_grad_(), randn((32,), 2).to(dev()).requires_grad_()
    y = api.linear_b128(x, w, b)
    assert y.shape == (0, 32)
    dx, dw, db = torch.autograd.grad(y, (x, w, b), torch.empty_like(y))
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


@pytest.mark.parametrize("M", [7, 300])
def test_step_calls_are_their_parts(M):
    """The two-call step gives bit for bit what its parts give, from views with
    strides, and can run backward twice."""
    N, K = 144, 272
    wide_x, wide_w, wide_d = spiky(M, K + 32, 1).to(dev()), spiky(N, K + 48, 2).to(dev()), randn((M, N + 24), 3).to(dev())
    x, w, dy, b = wide_x[:, 16:16 + K], wide_w[:, 8:8 + K], wide_d[:, 8:8 + N], randn((N,), 4).to(dev())
    leaves = [t.detach().requires_grad_() for t in (x, w, b)]
    y = api.linear_b128(*leaves)
    got = torch.autograd.grad(y, leaves, dy, retain_graph=True)
    again = torch.autograd.grad(y, leaves, dy)
    pw, pt = api.prepare_weight_b128_bf16(w)
    pa = api.quantize_act_packed_b128(x)
    db = torch.empty(N, dtype=torch.bfloat16, device=dev())
    dw, db = api.linear_wgrad(dy, pa, dtype=torch.bfloat16, bias_grad=True, out_bias=db)
    assert torch.equal(y, api.gemm_packed(pa, pw, b))
    for p, q, r in zip(got, (api.linear(dy, pt), dw, db), again):
        assert torch.equal(p, q) and torch.equal(p, r)


@pytest.mark.parametrize("M,N,K,form", [(70, 4104, 1040, "b128"), (30, 2600, 2064, "b128"), (130, 4224, 1024, "mx"),
                                        (700, 1032, 4240, "b128")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wgrad_several_tiles_per_workgroup(M, N, K, form, dtype):
    """More small tiles than compute units, of one to eleven steps: the copies
    of a workgroup's next tiles run ahead while it stores one, at the edges of
    the matrix too."""
    x, dy = spiky(M, K, M + K), randn((M, N), N, 1e-3)
    pa = keep(x, form)
    X = f64(pa.dequantize())
    base, base_b = torch.randn(N, K), torch.randn(N)
    prev = api.mxfp8_debug_force_wgrad(128)
    try:
        dw, db = api.linear_wgrad(dy.to(dev()), pa, dtype=dtype, bias_grad=True)
        again = api.linear_wgrad(dy.to(dev()), pa, dtype=dtype)
        acc = api.linear_wgrad(dy.to(dev()), pa, bias_grad=True, out=base.to(dev()), out_bias=base_b.to(dev()),
                               accumulate=True)
    finally:
        api.mxfp8_debug_force_wgrad(prev)
    check_dw(dw, db, dy, X)
    check_dw(*acc, dy, X, base, base_b)
    assert torch.equal(dw, again)


@pytest.mark.parametrize("M,N,K", [(16384, 64, 48), (9000, 256, 256), (5000, 136, 1040)])
def test_wgrad_tiles_of_many_runs(M, N, K):
    """Few tiles and many tokens: a tile in up to 128 pieces."""
    x, dy = spiky(M, K, 1), randn((M, N), 2, 1e-3)
    pa = keep(x, "b128")
    dw, db = api.linear_wgrad(dy.to(dev()), pa, bias_grad=True)
    check_dw(dw, db, dy, f64(pa.dequantize()))
    assert torch.equal(dw, api.linear_wgrad(dy.to(dev()), pa))
