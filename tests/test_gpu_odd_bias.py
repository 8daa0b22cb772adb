"""The bias of the tile GEMMs of the MXFP8 and W4A8 layers where N is odd, where the last tile holds few columns, and
where the bias starts between two words.  The weight is zero, so the output is the bias, exactly."""

import numpy as np
import pytest
import torch

import oracle
from mxfp8_block_scaled_amd import api, synth
from tests import gpu_util

pytestmark = pytest.mark.gpu

# (130 and 4: an even N beside the odd ones; 15300 rows: more tiles than workgroups)
SHAPES = [(200, 1, 256), (200, 3, 256), (200, 4, 256), (300, 127, 512), (300, 129, 768), (260, 130, 1024),
          (300, 255, 256), (513, 257, 512), (300, 383, 1024), (300, 385, 2048), (15300, 1281, 256)]


def zero_weight(kind, N, K):
    if kind == "mxfp8":
        return gpu_util.gpu_prepare(torch.zeros(N, K, dtype=torch.bfloat16))
    codes, s = oracle.quantize_mxfp4(np.zeros((N, K)))
    d = gpu_util.dev()
    return api.prepare_weight_fp4(torch.from_numpy(oracle.pack_fp4(codes)).to(d), torch.from_numpy(s).to(d))


def operands(M, N, K, start):
    g = torch.Generator().manual_seed(M + N)
    x = synth.randn_bf16((M, K), 1.0, g).to(gpu_util.dev())
    # what is around the bias is no bias
    around = torch.full((N + 8,), 1e4, dtype=torch.bfloat16)
    around[start:start + N] = synth.randn_bf16((N,), 1.0, g)
    return x, around.to(gpu_util.dev())[start:start + N]


def check(y, bias):
    torch.cuda.synchronize()
    off = (y != bias).nonzero()
    assert off.numel() == 0, (off.shape[0], off[0].tolist(), y[tuple(off[0])].item(), bias[off[0][1]].item())


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("kind", ["mxfp8", "w4a8"])
@pytest.mark.parametrize("start", [0, 1, 2])
def test_layer(M, N, K, kind, start):
    x, bias = operands(M, N, K, start)
    pw = zero_weight(kind, N, K)
    before = api.mxfp8_debug_force_path(17)      # tile GEMM, one K split: the persistent kernels
    try:
        y = api.linear(x, pw, bias)
    finally:
        api.mxfp8_debug_force_path(before)
    check(y, bias)


@pytest.mark.parametrize("M,N,K", [(513, 257, 512), (40, 1, 256)])
@pytest.mark.parametrize("start", [0, 1])
def test_packed_and_prequantized(M, N, K, start):
    x, bias = operands(M, N, K, start)
    pw = zero_weight("mxfp8", N, K)
    check(api.gemm_packed(api.quantize_act_packed(x), pw, bias), bias)
    q, s = api.quantize_act(x)
    check(api.gemm_prequant(q, s, pw, bias), bias)


@pytest.mark.parametrize("M", [1, 24, 100, 200, 1000, 3000])
@pytest.mark.parametrize("kind", ["mxfp8", "w4a8"])
def test_chosen_paths(M, kind):
    for N in (1001, 2049):
        x, bias = operands(M, N, 1024, 1)
        check(api.linear(x, zero_weight(kind, N, 1024), bias), bias)
