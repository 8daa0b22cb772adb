"""The linear layer with MXFP4 on both sides against its 64-bit form."""

import numpy as np
import pytest
import torch

import oracle
from mxfp8_block_scaled_amd import api
from tests import fp4_ref as ref
from tests import gpu_util

pytestmark = pytest.mark.gpu
dev = gpu_util.dev


def case(M, N, K, bias=True, form=0, seed=0):
    x = ref.activations(M, K, seed)
    packed, s, W = ref.weight(N, K, seed + 1)
    b = ref.activations(1, N, seed + 2, 0.1)[0] if bias else None
    pw = api.prepare_weight_fp4(torch.from_numpy(packed).to(dev()), torch.from_numpy(s).to(dev()))
    with ref.forced(form):
        y = api.linear_w4a4(x.to(dev()), pw, None if b is None else b.to(dev()))
        torch.cuda.synchronize()
    ref.check(y, ref.quantized(x), W, b)
    return x, pw, b, y


@pytest.mark.parametrize("M,K", [(1, 256), (5, 768), (128, 256), (130, 1024), (300, 2048)])
def test_quantize_packed(M, K):
    """Bytes of the packed quantizer: those of the row-major one, zero pad rows."""
    x = ref.activations(M, K, M)
    x[0, :32] = 0
    x[-1, 32:64] *= 2.0 ** -120
    x[0, 64:96] *= 2.0 ** 120
    pa = api.quantize_act_packed_fp4(x.to(dev()))
    q, s = pa.unpack()
    codes, sb = oracle.quantize_mxfp4(x.double().numpy())
    assert np.array_equal(q.cpu().numpy()[:M], oracle.pack_fp4(codes))
    assert np.array_equal(s.cpu().numpy()[:M], sb)
    assert bool((q[M:] == 0).all())


@pytest.mark.parametrize("form", [1, 2, 16, 64, 128, 256])
@pytest.mark.parametrize("M,N,K", [(1, 1, 256), (3, 130, 512), (16, 257, 768), (16, 1000, 2048), (9, 64, 4096), (2, 33, 8192),
                                   (17, 70, 256), (32, 100, 2048), (27, 300, 4096), (20, 64, 2304)])
def test_few_rows(form, M, N, K):
    case(M, N, K, form=form, seed=M + N)


@pytest.mark.parametrize("M,N,K", [(5, 30001, 512), (16, 13001, 2048), (9, 4500, 4096), (3, 4203, 8192), (20, 4401, 1024),
                                   (32, 4111, 4096)])
def test_runs_of_weight_blocks(M, N, K):
    """More blocks of 16 weight rows than the decode form's workgroups."""
    case(M, N, K, form=1, seed=M)


@pytest.mark.parametrize("M,N,K", [(33, 130, 256), (64, 200, 768), (65, 257, 2048), (100, 64, 4352), (128, 131, 8192),
                                   (50, 40, 12544), (128, 16, 20480)])
def test_mid_form(M, N, K):
    case(M, N, K, bias=(M % 2 == 1), form=16, seed=M)


@pytest.mark.parametrize("form", [2, 64, 128, 256])
@pytest.mark.parametrize("M,N,K", [(17, 128, 256), (64, 129, 512), (129, 131, 768), (300, 515, 1024), (513, 260, 1280),
                                   (1000, 1030, 512)])
def test_forms(form, M, N, K):
    case(M, N, K, bias=(M % 2 == 1), form=form, seed=M)


@pytest.mark.parametrize("form", [2, 64, 128, 256])
@pytest.mark.parametrize("K", [256, 512, 768])
def test_many_tiles_per_workgroup(form, K):
    """More tiles than workgroups: the copy stream runs over tile ends."""
    M, N = (2304, 8200) if form == 256 else (1500, 6500)
    case(M, N, K, bias=True, form=form, seed=K)


def test_chosen_forms():
    for M, N, K in [(1, 300, 9216), (17, 300, 1024), (200, 2056, 512), (2500, 1100, 256)]:
        case(M, N, K, seed=M)


@pytest.mark.parametrize("M", [4, 30, 128, 200])
def test_one_hot(M):
    """One-hot weights return single activations: every K position and row."""
    K, N = 512, 512
    x = ref.activations(M, K, 7)
    w = np.zeros((N, K))
    w[np.arange(N), (np.arange(N) * 37) % K] = 1.0
    codes, s = oracle.quantize_mxfp4(w)
    pw = api.prepare_weight_fp4(torch.from_numpy(oracle.pack_fp4(codes)).to(dev()), torch.from_numpy(s).to(dev()))
    A = ref.quantized(x)
    for form in (1, 2, 16, 64, 128, 256):
        with ref.forced(form):
            y = api.linear_w4a4(x.to(dev()), pw).double().cpu().numpy()
        assert np.array_equal(y, A[:, (np.arange(N) * 37) % K])


@pytest.mark.parametrize("form", [1, 2, 16, 64, 128, 256])
def test_not_finite(form):
    """An infinity or a NaN makes its own row's outputs NaN, and no other's."""
    M, N, K = 16, 200, 512
    x = ref.activations(M, K, 3)
    x[2, 5], x[4, 300], x[7, 511] = float("inf"), float("nan"), float("-inf")
    packed, s, W = ref.weight(N, K, 4)
    pw = api.prepare_weight_fp4(torch.from_numpy(packed).to(dev()), torch.from_numpy(s).to(dev()))
    with ref.forced(form):
        y = api.linear_w4a4(x.to(dev()), pw).cpu()
    bad = torch.zeros(M, dtype=torch.bool)
    bad[[2, 4, 7]] = True
    assert bool(torch.isnan(y[bad]).all())
    keep = (~bad).nonzero()[:, 0]
    ref.check(y[keep], ref.quantized(x[keep]), W)


@pytest.mark.parametrize("M", [5, 25, 90, 150])
def test_strides(M):
    """Rows of a wider matrix, unaligned rows, a strided and an unaligned output."""
    N, K = 264, 512
    packed, s, W = ref.weight(N, K, 1)
    pw = api.prepare_weight_fp4(torch.from_numpy(packed).to(dev()), torch.from_numpy(s).to(dev()))
    wide = ref.activations(M, K + 24, 2)
    b = ref.activations(1, N + 1, 3)[0]
    for lo in (8, 3):
        x = wide[:, lo:lo + K]
        want = ref.quantized(x)
        buf = torch.full((M, N + 16), 7.0, dtype=torch.bfloat16, device=dev())
        for at in (8, 1):
            out = buf[:, at:at + N]
            api.linear_w4a4(wide.to(dev())[:, lo:lo + K], pw, b.to(dev())[1:], out=out)
            ref.check(out, want, W, b[1:])
            assert bool((buf[:, :at] == 7).all()) and bool((buf[:, at + N:] == 7).all())
            buf.fill_(7.0)


def test_shapes_and_empty():
    packed, s, W = ref.weight(130, 256, 1)
    pw = api.prepare_weight_fp4(torch.from_numpy(packed).to(dev()), torch.from_numpy(s).to(dev()))
    x = ref.activations(6, 256, 2)
    y = api.linear_w4a4(x.to(dev()).view(2, 3, 256), pw)
    assert y.shape == (2, 3, 130)
    ref.check(y.view(6, 130), ref.quantized(x), W)
    y = api.linear_w4a4(x.to(dev())[0], pw)
    assert y.shape == (130,)
    assert api.linear_w4a4(x.to(dev())[:0], pw).shape == (0, 130)
    y += 1   # an output of its own


def test_packed_product_matches_layer():
    M, N, K = 300, 520, 512
    x = ref.activations(M, K, 1).to(dev())
    packed, s, _ = ref.weight(N, K, 2)
    pw = api.prepare_weight_fp4(torch.from_numpy(packed).to(dev()), torch.from_numpy(s).to(dev()))
    pa = api.quantize_act_packed_fp4(x)
    assert torch.equal(api.gemm_packed(pa, pw), api.linear_w4a4(x, pw))
    with pytest.raises(ValueError):
        api.gemm_packed(api.quantize_act_packed(x), pw)
    with pytest.raises(ValueError):
        api.gemm_packed(pa, api.prepare_weight(*api.quantize_act(x)))


@pytest.mark.parametrize("M", [3, 700])
def test_captured(M):
    """A captured call replayed on new rows, on a side stream."""
    N, K = 520, 1024
    packed, s, W = ref.weight(N, K, 2)
    pw = api.prepare_weight_fp4(torch.from_numpy(packed).to(dev()), torch.from_numpy(s).to(dev()))
    x = ref.activations(M, K, 1).to(dev())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        api.linear_w4a4(x, pw)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = api.linear_w4a4(x, pw)
    for seed in (5, 6, 7):
        x.copy_(ref.activations(M, K, seed))
        graph.replay()
        want = api.linear_w4a4(x, pw)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
