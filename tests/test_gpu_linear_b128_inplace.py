"""The 128-block layer's output changed in place, as a residual is added to it:
for every number of leading dimensions, gradients as without."""

import pytest
import torch

from mxfp8_block_scaled_amd import api
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

N, K = 144, 272


@pytest.mark.parametrize("lead", [(), (5,), (1, 7), (2, 33), (2, 3, 50)])
def test_output_changed_in_place(lead):
    g = torch.Generator().manual_seed(len(lead))
    x, w, b, r, dy = (torch.randn(s, generator=g).to(torch.bfloat16).to(dev())
                      for s in (lead + (K,), (N, K), (N,), lead + (N,), lead + (N,)))
    operands = [t.requires_grad_() for t in (x, w, b)]
    plain = api.linear_b128(*operands)
    want = torch.autograd.grad(plain, operands, dy)
    y = api.linear_b128(*operands)
    assert y.shape == lead + (N,) and y.is_contiguous()
    y += r
    assert torch.equal(y, plain + r)
    for p, q in zip(torch.autograd.grad(y, operands, dy), want):
        assert torch.equal(p, q)
