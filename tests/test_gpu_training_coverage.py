"""Forms of the training operators that no size of the other tests reaches:
more than eight experts per token where a lane holds several logits, and the
large tiles of the weight gradient on a slice of a wider dY."""

import pytest
import torch

from mxfp8_block_scaled_amd import api
from tests.gpu_util import dev
from tests.test_gpu_b128 import f64, randn, spiky
from tests.test_gpu_balance import check, make
from tests.test_gpu_wgrad import check_dw, keep

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(30, 9), (60, 16), (64, 11), (100, 16), (128, 9), (200, 13), (256, 16)])
def test_many_experts_per_token(E, k, dtype):
    check(make(77, E, E + k, dtype), k)
    # logits from a handful of values: nearly every selection ends in a tie
    check(make(300, E, E - k, dtype, spread=0.7).round(), k)


@pytest.mark.parametrize("form", ["mx", "b128"])
@pytest.mark.parametrize("M,accumulate", [(190, False), (64, True), (1, True)])
def test_large_tiles_on_a_slice(form, M, accumulate):
    """The slice's neighbours are NaN and its output's are kept."""
    N, K = 264, 512
    pa = keep(spiky(M, K, 1), form)
    X = f64(pa.dequantize())
    wide = torch.full((M, N + 64), float("nan"), dtype=torch.bfloat16, device=dev())
    wide[:, 32:32 + N] = randn((M, N), 2).to(dev())
    dy = wide[:, 32:32 + N]
    out = torch.full((N + 2, K + 16), 5.0, device=dev())
    db = torch.full((N,), 5.0, device=dev())
    base = (out[1:N + 1, :K].cpu(), db.cpu()) if accumulate else (None, None)
    old = api.mxfp8_debug_force_wgrad(256)
    try:
        dw, db = api.linear_wgrad(dy, pa, bias_grad=True, out=out[1:N + 1, :K], out_bias=db, accumulate=accumulate)
    finally:
        api.mxfp8_debug_force_wgrad(old)
    check_dw(dw, db, dy.cpu(), X, *base)
    edge = out.clone()
    edge[1:N + 1, :K] = 5.0
    assert (edge == 5.0).all()
