"""Rows there and back with results larger than 32 MiB, whose stores go around the caches, against plain 64-bit forms:
each element type with rows on 16 bytes and off them; and long rows of few tokens."""

import pytest
import torch

from mxfp8_block_scaled_amd import api
from tests import gpu_util
from tests.test_gpu_moe_order import close, inputs, sort_ref

pytestmark = pytest.mark.gpu
dev = gpu_util.dev


@pytest.mark.parametrize("T,topk,E,H,dtype", [
    (2500, 4, 60, 1003, torch.float32), (2500, 4, 60, 1004, torch.float32), (4500, 4, 60, 1003, torch.bfloat16),
    (4500, 4, 60, 1008, torch.bfloat16), (2100, 9, 16, 1001, torch.bfloat16), (4300, 2, 8, 1001, torch.float32),
    # four waves per token in the gradient
    (900, 3, 8, 7003, torch.bfloat16), (900, 3, 8, 4096, torch.float32), (1500, 4, 8, 4096, torch.bfloat16),
    (700, 2, 8, 6001, torch.float32)])
def test_there_and_back(T, topk, E, H, dtype):
    drop = 0.3
    assert T * topk * H * dtype.itemsize > 32 << 20
    ids, x, ys, w, dxs, dy = inputs(T, topk, E, H, dtype, T, drop)
    rows, slots, offsets = (t.to(dev()) for t in sort_ref(ids, E))
    kept = int(offsets[E])
    eps = torch.finfo(dtype).eps if dtype != torch.float32 else 0.0
    x, ys, w, dxs, dy = (t.to(dev()) for t in (x, ys, w, dxs, dy))
    order = api.moe_sort(ids.to(dev()), E)
    xg, yg, wg = (t.clone().requires_grad_() for t in (x, ys, w))
    xs = api.moe_permute(xg, order)
    y = api.moe_unpermute(yg, order, wg)
    gx, gy, gw = torch.autograd.grad((xs, y), (xg, yg, wg), (dxs, dy))

    token = slots // topk
    assert torch.equal(xs[:kept], x[token[:kept]]) and bool((xs[kept:] == 0).all())
    here = (rows < kept).double()[:, :, None]
    by_slot = ys.double()[rows.reshape(-1)].view(T, topk, H) * here
    ww = w.double()[:, :, None]
    close(y, (ww * by_slot).sum(1).cpu(), eps, topk, (ww * by_slot.abs()).sum(1).cpu())
    prod = by_slot * dy.double()[:, None, :]
    close(gw, prod.sum(2).cpu(), 0.0, H, prod.abs().sum(2).cpu())
    back = dxs.double()[rows.reshape(-1)].view(T, topk, H) * here
    close(gx, back.sum(1).cpu(), eps, topk, back.abs().sum(1).cpu())
    want = (w.double() * here[:, :, 0]).reshape(-1)[slots][:, None] * dy.double()[token]
    close(gy, want.cpu(), eps, 1, want.abs().cpu())
    assert bool((gy[kept:] == 0).all()) and bool((gw[here[:, :, 0] == 0] == 0).all())
    # one gradient alone
    y = api.moe_unpermute(ys, order, wg)
    assert torch.equal(torch.autograd.grad(y, wg, dy)[0], gw)
    y = api.moe_unpermute(yg, order, w)
    assert torch.equal(torch.autograd.grad(y, yg, dy)[0], gy)
