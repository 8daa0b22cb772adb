"""The experts' MXFP4 products on sorted rows against their 64-bit form."""

import numpy as np
import pytest
import torch

from mxfp8_block_scaled_amd import api
from tests import fp4_ref as ref
from tests import gpu_util
from tests.test_gpu_moe_order import make_ids, sort_ref

pytestmark = pytest.mark.gpu
dev = gpu_util.dev


def experts(E, N, K, seed):
    parts = [ref.weight(N, K, seed + e) for e in range(E)]
    return np.stack([p[0] for p in parts]), np.stack([p[1] for p in parts]), [p[2] for p in parts]


def case(T, topk, E, N, K, gather, form=0, drop=0.0, seed=0, ids=None):
    ids = make_ids(T, topk, E, seed, drop) if ids is None else ids
    packed, s, W = experts(E, N, K, seed)
    x = ref.activations(T if gather else T * topk, K, seed + 1)
    order = api.moe_sort(ids.to(dev()), E)
    ew = api.moe_prepare_experts_fp4(torch.from_numpy(packed).to(dev()), torch.from_numpy(s).to(dev()))
    with ref.forced(form):
        y = api.moe_linear_w4a4(x.to(dev()), ew, order, gather=gather)
        torch.cuda.synchronize()
    _, slots, offsets = sort_ref(ids, E)
    A = ref.quantized(x)
    if gather:
        A = A[(slots // topk).numpy()]
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b > a:
            ref.check(y[a:b], A[a:b], W[e])
    assert bool((y[int(offsets[E]):] == 0).all())


FORMS = [1, 2, 64, 128, 256]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("T,topk,E,N,K", [(1, 1, 1, 1, 256), (1, 8, 16, 130, 256), (20, 2, 5, 100, 512),
                                          (70, 3, 4, 300, 768), (300, 4, 7, 257, 1024), (129, 1, 1, 520, 2048)])
def test_forms(form, gather, T, topk, E, N, K):
    case(T, topk, E, N, K, gather, form, drop=0.3 if T % 2 == 0 else 0.0, seed=T)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("K", [256, 512, 768])
def test_many_tiles_per_workgroup(form, K):
    case(1500, 4, 24, 1100, K, True, form, drop=0.1, seed=K)


@pytest.mark.parametrize("T,topk,E,N,K", [(100, 8, 40, 901, 512), (40, 4, 40, 420, 1536), (30, 3, 8, 530, 4096),
                                          (20, 2, 3, 1401, 8192)])
@pytest.mark.parametrize("gather", [True, False])
def test_runs_of_weight_blocks(T, topk, E, N, K, gather):
    """More blocks of 16 weight rows than the decode form's workgroups, experts with more rows than 16, and none."""
    case(T, topk, E, N, K, gather, 1, drop=0.2, seed=K)


@pytest.mark.parametrize("form", FORMS)
def test_unusual_orders(form):
    """One expert for all, none at all, the last expert only, the same expert twice in a token."""
    case(150, 2, 6, 140, 512, True, form, ids=torch.full((150, 2), 5))
    case(150, 2, 6, 140, 512, False, form, ids=torch.full((150, 2), 0))
    case(10, 2, 6, 140, 512, True, form, ids=torch.full((10, 2), -1))
    case(40, 4, 6, 140, 512, True, form, ids=torch.randint(0, 6, (40, 4), generator=torch.Generator().manual_seed(2)))


def test_chosen_forms():
    for T, topk, E, N, K in [(2, 8, 64, 96, 256), (300, 2, 8, 200, 512), (700, 4, 16, 264, 9216), (2, 1, 3, 64, 9216)]:
        case(T, topk, E, N, K, True, seed=T)


def test_256_experts():
    case(500, 8, 256, 72, 256, True, 0, seed=5)
    case(500, 8, 256, 72, 256, False, 128, seed=5)


@pytest.mark.parametrize("form", FORMS)
def test_not_finite(form):
    """An infinite token makes its own rows NaN, and no other's; one without an expert nothing."""
    T, topk, E, N, K = 50, 2, 4, 130, 512
    ids = make_ids(T, topk, E, 1)
    ids[9] = -1
    packed, s, _ = experts(E, N, K, 1)
    x = ref.activations(T, K, 2)
    ew = api.moe_prepare_experts_fp4(torch.from_numpy(packed).to(dev()), torch.from_numpy(s).to(dev()))
    order = api.moe_sort(ids.to(dev()), E)
    with ref.forced(form):
        clean = api.moe_linear_w4a4(x.to(dev()), ew, order, gather=True)
        x[3, 100], x[9, 5] = float("inf"), float("nan")
        y = api.moe_linear_w4a4(x.to(dev()), ew, order, gather=True)
    bad = torch.zeros(T * topk, dtype=torch.bool, device=dev())
    bad[order.rows[3].long()] = True
    assert bool(torch.isnan(y[bad]).all()) and torch.equal(y[~bad], clean[~bad])


def test_run_together():
    """A routed layer from its parts: sort, first product from the tokens, gate, second product, back; each part
    against its 64-bit form on what the part before it gave."""
    T, topk, E, H, I = 200, 4, 12, 512, 256
    g = torch.Generator().manual_seed(3)
    logits = torch.randn(T, E, generator=g).to(dev())
    top, ids = torch.topk(logits, topk, dim=1)
    weights = torch.softmax(top, dim=1)
    p13, s13, W13 = experts(E, 2 * I, H, 10)
    p2, s2, W2 = experts(E, H, I, 50)
    w13 = api.moe_prepare_experts_fp4(torch.from_numpy(p13).to(dev()), torch.from_numpy(s13).to(dev()))
    w2 = api.moe_prepare_experts_fp4(torch.from_numpy(p2).to(dev()), torch.from_numpy(s2).to(dev()))
    x = ref.activations(T, H, 4).to(dev())

    def layer():
        order = api.moe_sort(ids, E)
        h = api.moe_linear_w4a4(x, w13, order, gather=True)
        act = (torch.nn.functional.silu(h[:, :I].float()) * h[:, I:].float()).to(torch.bfloat16)
        ys = api.moe_linear_w4a4(act, w2, order)
        return order, h, act, ys, api.moe_unpermute(ys, order, weights)

    order, h, act, ys, y = layer()
    _, slots, offsets = sort_ref(ids.cpu(), E)
    assert torch.equal(h, api.moe_linear_w4a4(api.moe_permute(x, order), w13, order))
    A, B = ref.quantized(x.cpu())[(slots // topk).numpy()], ref.quantized(act.cpu())
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b > a:
            ref.check(h[a:b], A[a:b], W13[e])
            ref.check(ys[a:b], B[a:b], W2[e])
    rows = order.rows.long()
    want = (weights.double()[:, :, None] * ys.double()[rows.view(-1)].view(T, topk, H)).sum(1)
    scale = (weights.double()[:, :, None] * ys.double()[rows.view(-1)].view(T, topk, H).abs()).sum(1)
    assert bool(((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * scale).all())
    # captured and replayed
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()[-1]
    for seed in (7, 8, 9):
        x.copy_(ref.activations(T, H, seed))
        ids.copy_(torch.topk(torch.randn(T, E, generator=g), topk, dim=1).indices)
        graph.replay()
        again = layer()[-1]
        torch.cuda.synchronize()
        assert torch.equal(out, again)
