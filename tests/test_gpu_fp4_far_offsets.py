"""Byte and element offsets past 32 bits in the MXFP4 layer, the experts'
products and the rows there and back.  Far rows and columns are checked
against plain forms of those alone."""

import numpy as np
import pytest
import torch

import oracle
from mxfp8_block_scaled_amd import api
from tests import fp4_ref as ref
from tests import gpu_util
from tests.test_gpu_far_offsets import far_rows
from tests.test_gpu_moe_order import close, make_ids, sort_ref

pytestmark = pytest.mark.gpu
dev = gpu_util.dev


def values(packed, s):
    """What row-major codes [n, K/2] and scale bytes [n, K/32] (GPU) are worth."""
    return oracle.dequantize_mxfp4(packed.cpu().numpy(), s.cpu().numpy())


def random_weight(rows, K, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    w = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device=dev(), generator=g)
    return w, torch.randint(118, 123, (rows, K // 32), dtype=torch.uint8, device=dev(), generator=g)


def test_layer_of_many_tokens():
    M, N, K = 1_100_000, 136, 8192          # x 18 GB, its codes 4.5 GB
    rows = torch.unique(torch.cat([far_rows(M, 2 * K), far_rows(M, K // 2)]))
    xs = ref.activations(len(rows), K, 1)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=dev())
    x[rows.to(dev())] = xs.to(dev())
    packed, s, W = ref.weight(N, K, 2)
    pw = api.prepare_weight_fp4(torch.from_numpy(packed).to(dev()), torch.from_numpy(s).to(dev()))
    A = ref.quantized(xs)
    pa = api.quantize_act_packed_fp4(x)
    assert pa.q_packed.numel() > 1 << 32
    for form in (64, 128, 256):
        with ref.forced(form):
            y = api.gemm_packed(pa, pw)
        ref.check(y[rows.to(dev())], A, W)
        assert int((y != 0).any(dim=1).sum()) == len(rows)
    del pa
    y = api.linear_w4a4(x, pw)
    ref.check(y[rows.to(dev())], A, W)


@pytest.mark.parametrize("form", [2, 64, 128, 256])
def test_layer_with_a_large_result(form):
    M, N, K = 300_000, 8200, 256            # y 4.9 GB
    x = ref.activations(M, K, 3)
    packed, s, W = ref.weight(N, K, 4)
    pw = api.prepare_weight_fp4(torch.from_numpy(packed).to(dev()), torch.from_numpy(s).to(dev()))
    with ref.forced(form):
        y = api.linear_w4a4(x.to(dev()), pw)
    rows = far_rows(M, 2 * N)
    ref.check(y[rows.to(dev())], ref.quantized(x[rows]), W)


@pytest.mark.parametrize("form", [1, 2, 16, 64, 128, 256])
def test_far_apart_rows(form):
    """Rows of x and y 268 MB apart."""
    M, N, K = 16, 200, 1024
    wide = torch.zeros(M + 1, (1 << 27) + 8, dtype=torch.bfloat16, device=dev())
    x = ref.activations(M, K, 5)
    wide[:M, :K] = x.to(dev())
    packed, s, W = ref.weight(N, K, 6)
    pw = api.prepare_weight_fp4(torch.from_numpy(packed).to(dev()), torch.from_numpy(s).to(dev()))
    with ref.forced(form):
        api.linear_w4a4(wide[:M, :K], pw, out=wide[:M, K:K + N])
    ref.check(wide[:M, K:K + N], ref.quantized(x), W)
    assert bool((wide[M] == 0).all()) and bool((wide[:M, K + N:K + N + 512] == 0).all())


def test_layer_with_a_large_weight():
    N, K = 1_050_000, 8192                  # 4.3 GB of codes
    w, s = random_weight(N, K, 7)
    pw = api.prepare_weight_fp4(w, s)
    cols = far_rows(N, K // 2).to(dev())
    W = values(w[cols], s[cols])
    del w
    for M, form in ((3, 1), (40, 16), (70, 64), (140, 128), (300, 256)):
        x = ref.activations(M, K, M)
        with ref.forced(form):
            y = api.linear_w4a4(x.to(dev()), pw)
        ref.check(y[:, cols], ref.quantized(x), W)


def test_experts_with_large_weights():
    E, N, K, T, topk = 64, 16500, 8192, 60, 8   # 4.3 GB of codes
    w, s = random_weight(E * N, K, 8)
    ew = api.moe_prepare_experts_fp4(w.view(E, N, K // 2), s.view(E, N, K // 32))
    ids = make_ids(T, topk, E, 9)
    ids[0] = torch.arange(E - topk, E)
    order = api.moe_sort(ids.to(dev()), E)
    _, slots, offsets = sort_ref(ids, E)
    x = ref.activations(T, K, 10)
    A = ref.quantized(x)
    cols = torch.tensor([0, 1, 127, 128, 8191, N - 2, N - 1], device=dev())
    some = [(e, values(w[e * N + cols], s[e * N + cols])) for e in (0, 31, 32, 62, 63)]
    del w
    for form in (1, 64, 128, 256):
        with ref.forced(form):
            y = api.moe_linear_w4a4(x.to(dev()), ew, order, gather=True)
        for e, W in some:
            a, b = int(offsets[e]), int(offsets[e + 1])
            if b > a:
                ref.check(y[a:b][:, cols], A[(slots[a:b] // topk).numpy()], W)


@pytest.mark.parametrize("form", [1, 2, 64, 128, 256])
def test_experts_with_a_large_result(form):
    T, topk, E, N, K = 40_000, 8, 8, 8200, 256  # y 5.2 GB
    ids = make_ids(T, topk, E, 11, 0.05)
    parts = [ref.weight(N, K, 12 + e) for e in range(E)]
    ew = api.moe_prepare_experts_fp4(*(torch.from_numpy(np.stack([p[i] for p in parts])).to(dev()) for i in (0, 1)))
    order = api.moe_sort(ids.to(dev()), E)
    _, slots, offsets = sort_ref(ids, E)
    x = ref.activations(T, K, 30)
    with ref.forced(form):
        y = api.moe_linear_w4a4(x.to(dev()), ew, order, gather=True)
    kept = int(offsets[E])
    rows = torch.unique(torch.cat([far_rows(T * topk, 2 * N), torch.tensor([kept - 1])]))
    for r in rows[rows < kept].tolist():
        e = int((offsets[1:] <= r).sum())
        ref.check(y[r:r + 1], ref.quantized(x[slots[r] // topk][None]), parts[e][2])
    assert not bool(y[kept:].any())


@pytest.mark.parametrize("T,topk", [(300_000, 1), (40_000, 8)])
def test_rows_there_and_back(T, topk):
    H, E = 8192, 16                         # [T topk, H]: 4.9 and 5.2 GB
    ids = make_ids(T, topk, E, 13, 0.02)
    rows, slots, offsets = sort_ref(ids, E)
    kept = int(offsets[E])
    order = api.moe_sort(ids.to(dev()), E)
    g = torch.Generator(device=dev()).manual_seed(14)
    rand = lambda n: torch.randn(n, H, dtype=torch.bfloat16, device=dev(), generator=g)
    x = rand(T)
    xs = api.moe_permute(x, order)
    far = far_rows(T * topk, 2 * H)
    for r in far.tolist() + [kept - 1, kept]:
        assert torch.equal(xs[r], x[slots[r] // topk] if r < kept else torch.zeros_like(xs[r]))
    del xs
    ys = rand(T * topk).requires_grad_()
    w = torch.rand(T, topk, device=dev(), generator=g).requires_grad_()
    y = api.moe_unpermute(ys, order, w)
    dys, dw = torch.autograd.grad(y, (ys, w), x)
    tokens = torch.unique(torch.cat([slots[far] // topk, far_rows(T, 2 * H)]))
    eps = torch.finfo(torch.bfloat16).eps
    here = (rows[tokens] < kept).double()[:, :, None]
    at = rows[tokens].to(dev())
    by_slot, ww, dy = ys.detach()[at].double().cpu() * here, w.detach().cpu().double()[tokens][:, :, None], x[tokens.to(dev())].double().cpu()
    close(y[tokens.to(dev())].detach(), (ww * by_slot).sum(1), eps, topk, (ww * by_slot.abs()).sum(1))
    want = here * ww * dy[:, None]
    close(dys[at], want, eps, 1, want.abs())
    prod = by_slot * dy[:, None]
    close(dw[tokens.to(dev())], prod.sum(2), 0.0, H, prod.abs().sum(2))
