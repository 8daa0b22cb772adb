"""The MXFP4 layer, the sort, the rows there and back and the experts' products
on several streams at once and in several captured graphs, against the same
calls one at a time."""

import pytest
import torch

from mxfp8_block_scaled_amd import api
from tests import fp4_ref as ref
from tests import gpu_util
from tests.test_gpu_moe_order import make_ids

pytestmark = pytest.mark.gpu
dev = gpu_util.dev


def operands(seed):
    T, topk, E, N, K = 900, 4, 24, 520, 1024
    packed, s, _ = ref.weight(E * N, K, seed)
    w, s = torch.from_numpy(packed).to(dev()), torch.from_numpy(s).to(dev())
    return dict(ids=make_ids(T, topk, E, seed, 0.1).to(dev()), E=E, x=ref.activations(T, K, seed + 1).to(dev()),
                weights=torch.rand(T, topk, generator=torch.Generator().manual_seed(seed)).to(dev()),
                pw=api.prepare_weight_fp4(w, s),
                ew=api.moe_prepare_experts_fp4(w.view(E, N, K // 2), s.view(E, N, K // 32)))


def step(o):
    order = api.moe_sort(o["ids"], o["E"])
    xs = api.moe_permute(o["x"], order)
    ys = api.moe_linear_w4a4(xs, o["ew"], order)
    return api.moe_unpermute(ys, order, o["weights"]), api.linear_w4a4(o["x"], o["pw"])


@pytest.mark.parametrize("form", [0, 64, 128, 256])
def test_streams_at_once(form):
    cases = [operands(s) for s in (1, 2, 3)]
    with ref.forced(form):
        want = [step(o) for o in cases]
        streams = [torch.cuda.Stream() for _ in cases]
        torch.cuda.synchronize()
        got = []
        for turn in range(4):
            for o, st in zip(cases, streams):
                with torch.cuda.stream(st):
                    got.append(step(o))
        torch.cuda.synchronize()
    for i, outs in enumerate(got):
        for a, b in zip(outs, want[i % 3]):
            assert torch.equal(a, b)


def test_two_captured_graphs():
    """Replayed in turns and side by side on two streams."""
    cases = [operands(s) for s in (4, 5)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), ref.forced(128):
        for o in cases:
            step(o)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    with ref.forced(128):
        for o in cases:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                outs.append(step(o))
    streams = [torch.cuda.Stream() for _ in cases]
    for turn in range(3):
        for o in cases:
            o["x"].add_(0.5)
        with ref.forced(128):
            want = [step(o) for o in cases]
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_results_may_be_changed_in_place():
    o = operands(6)
    order = api.moe_sort(o["ids"], o["E"])
    x = o["x"].clone().requires_grad_()
    y = api.moe_unpermute(api.moe_permute(x, order), order, o["weights"])
    y.mul_(2.0).add_(1.0)
    y.sum().backward()
    x2 = o["x"].clone().requires_grad_()
    y2 = 2.0 * api.moe_unpermute(api.moe_permute(x2, order), order, o["weights"]) + 1.0
    y2.sum().backward()
    assert torch.equal(y.detach(), y2.detach()) and torch.equal(x.grad, x2.grad)


def test_no_rows():
    p = api.quantize_act_packed_fp4(torch.empty(0, 512, dtype=torch.bfloat16, device=dev()))
    packed, s, _ = ref.weight(64, 512, 1)
    pw = api.prepare_weight_fp4(torch.from_numpy(packed).to(dev()), torch.from_numpy(s).to(dev()))
    assert api.gemm_packed(p, pw).shape == (0, 64)
    codes, scales = p.unpack()
    assert codes.shape == (0, 256) and scales.shape == (0, 16)
