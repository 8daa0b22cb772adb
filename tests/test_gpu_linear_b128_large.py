"""The training step where its GEMMs run on the MXFP8 tile GEMM (whole rounds of
256 x 256 tiles, the summed axis a multiple of 256): sampled rows against
64-bit forms, and the other combinations of forward and backward forms."""

import numpy as np
import pytest
import torch

from mxfp8_block_scaled_amd import api
from tests import b128_ref as ref
from tests.gpu_util import dev
from tests.test_gpu_b128 import f64, randn, spiky
from tests.test_gpu_wgrad import check_close, check_dw

pytestmark = pytest.mark.gpu

# forward and dX on the MX GEMM; forward only; dX only (N and K change places); ragged M and N
SHAPES = [(8192, 2048, 2048), (4096, 4096, 256), (4096, 256, 4096), (8000, 2032, 2048)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_large_step(M, N, K):
    x, w, b, dy = spiky(M, K, 1), spiky(N, K, 2), randn((N,), 3), spiky(M, N, 4)
    leaves = [t.to(dev()).requires_grad_() for t in (x, w, b)]
    y = api.linear_b128(*leaves)
    dx, dw, db = torch.autograd.grad(y, leaves, dy.to(dev()))
    rows = torch.cat([torch.arange(40), torch.arange(M - 200, M, 7), torch.randint(M, (60,))])
    _, _, A = ref.quantize(f64(x[rows]))
    _, _, D = ref.quantize(f64(dy[rows]))
    _, _, W = ref.quantize(f64(w), rows=128)
    check_close(y[rows.to(dev())], A @ W.T + f64(b), ref.gemm_bound(A, W))
    check_close(dx[rows.to(dev())], D @ W, ref.gemm_bound(D, W.T))
    pa = api.quantize_act_packed_b128(x.to(dev()))
    same = api.linear_wgrad(dy.to(dev()), pa, dtype=torch.bfloat16)
    assert torch.equal(dw, same)
    # every row: the 128-block GEMM on the same operands is within both bounds
    pw, pt = api.prepare_weight_b128_bf16(w.to(dev()))
    for got, want in ((y, api.gemm_packed(pa, pw, b.to(dev()))),
                      (dx, api.gemm_packed(api.quantize_act_packed_b128(dy.to(dev())), pt))):
        got, want = got.float(), want.float()
        assert ((got - want).norm() / want.norm()) < 2.0 ** -7
    with torch.no_grad():   # nothing kept: the same GEMM
        assert torch.equal(api.linear_b128(*leaves), y)


def test_large_step_non_finite():
    """A non-finite weight block makes its outputs NaN and no others, through
    scales in either layout."""
    M, N, K = 8192, 2048, 2048
    x, w, dy = randn((M, K), 1), randn((N, K), 2, 0.02), randn((M, N), 3)
    w[130, 300] = float("inf")
    x[77, 5] = float("nan")
    leaves = [t.to(dev()).requires_grad_() for t in (x, w)]
    y = api.linear_b128(*leaves)
    dx, = torch.autograd.grad(y, leaves[:1], dy.to(dev()))
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[:, 128:256] = True     # the rows of the block in W
    bad[77] = True
    assert torch.equal(torch.isnan(y).cpu(), bad)
    bad = torch.zeros(M, K, dtype=torch.bool)
    bad[:, 256:384] = True     # its columns
    assert torch.equal(torch.isnan(dx).cpu(), bad)
