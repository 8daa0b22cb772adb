"""Byte and element offsets past 32 bits: many tokens through the 128-block
layer, the weight gradient and the balance loss.  Far rows are checked against
plain forms of those rows alone."""

import numpy as np
import pytest
import torch

from mxfp8_block_scaled_amd import api
from tests import b128_ref as ref
from tests.gpu_util import dev
from tests.test_gpu_b128 import f64, randn, spiky

pytestmark = pytest.mark.gpu


def far_rows(M, row_bytes):
    """The first and last rows and those around 2^31 and 2^32 bytes."""
    at = {0, 1, M - 2, M - 1}
    for b in (1 << 31, 1 << 32):
        at |= {b // row_bytes - 1, b // row_bytes, b // row_bytes + 1}
    return torch.tensor(sorted(r for r in at if 0 <= r < M))


def test_layer_and_gradient_of_many_tokens():
    M, N, K = 1_100_000, 136, 4096   # x 9.0 GB, its checkpoint 4.5 GB
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=dev())
    rows = torch.unique(torch.cat([far_rows(M, 2 * K), far_rows(M, K)]))
    xs = spiky(len(rows), K, 5)
    x[rows.to(dev())] = xs.to(dev())
    w = randn((N, K), 6, 0.02)
    pw, _ = api.prepare_weight_b128_bf16(w.to(dev()), transposed=False)
    pa = api.quantize_act_packed_b128(x)
    assert pa.q_packed.numel() > 1 << 32
    y = api.gemm_packed(pa, pw)
    _, _, A = ref.quantize(f64(xs))
    _, _, W = ref.quantize(f64(w), rows=128)
    want = A @ W.T
    err = np.abs(f64(y[rows.to(dev())]) - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + ref.gemm_bound(A, W)).all()
    assert int((y != 0).any(dim=1).sum()) == len(rows)   # the rows of zeros stay zeros
    back = pa.dequantize()
    assert np.array_equal(f64(back[rows.to(dev())]), A)
    del back, x
    # dW: only these tokens' rows of dY are set
    dy = torch.zeros(M, N, dtype=torch.bfloat16, device=dev())
    ds = randn((len(rows), N), 7, 1e-2)
    dy[rows.to(dev())] = ds.to(dev())
    dw, db = api.linear_wgrad(dy, pa, bias_grad=True)
    want, mag = f64(ds).T @ A, np.abs(f64(ds)).T @ np.abs(A)
    # zeros add exactly: the additions that round are the rows' and the joins'
    assert (np.abs(f64(dw) - want) <= (len(rows) + 600) * 2.0 ** -23 * mag).all()
    assert (np.abs(f64(db) - f64(ds).sum(0)) <= (len(rows) + 600) * 2.0 ** -23 * np.abs(f64(ds)).sum(0)).all()


def test_wide_dy_of_many_tokens():
    M, N, K = 600_000, 4096, 48      # dY 4.9 GB
    rows = torch.unique(far_rows(M, 2 * N))
    xs, ds = spiky(len(rows), K, 8), randn((len(rows), N), 9, 1e-2)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=dev())
    dy = torch.zeros(M, N, dtype=torch.bfloat16, device=dev())
    x[rows.to(dev())] = xs.to(dev())
    dy[rows.to(dev())] = ds.to(dev())
    _, _, A = ref.quantize(f64(xs))
    for tile in (128, 256):
        prev = api.mxfp8_debug_force_wgrad(tile)
        try:
            dw = api.linear_wgrad(dy, api.quantize_act_packed_b128(x))
        finally:
            api.mxfp8_debug_force_wgrad(prev)
        mag = np.abs(f64(ds)).T @ np.abs(A)
        assert (np.abs(f64(dw) - f64(ds).T @ A) <= (len(rows) + 600) * 2.0 ** -23 * mag).all()


def test_balance_of_many_tokens():
    T, E = 20_000_000, 128           # 5.1 GB
    logits = torch.zeros(T, E, dtype=torch.bfloat16, device=dev())
    t = torch.arange(T, device=dev())
    logits[t, t % E] = 4.0
    loss, counts, used = api.moe_balance(logits, 1, coef=1.0)
    assert int(used) == T
    assert torch.equal(counts, torch.bincount(t % E, minlength=E).to(torch.int32))
    # equal shares but for T % E: the loss of a balanced router is coef = 1
    assert abs(float(loss) - 1.0) < 1e-5
    rows = far_rows(T, 2 * E).to(dev())
    skew = torch.randint(1, 1000, (E,), dtype=torch.int32, device=dev())
    d = api.moe_balance_backward(logits, 1, skew, used, coef=1e6)
    want = api.moe_balance_backward(logits[rows].contiguous(), 1, skew, used, coef=1e6)
    assert torch.equal(d[rows], want)
