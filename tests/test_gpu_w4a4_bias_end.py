"""The end of linear_w4a4's bias where N is odd: its last value is added, and what shares a word with it (the kernels
read whole words) reaches no output, in every form.  The weight is zero, so the output is the bias, exactly."""

import numpy as np
import pytest
import torch

import oracle
from mxfp8_block_scaled_amd import api, synth
from tests import fp4_ref as ref
from tests import gpu_util

pytestmark = pytest.mark.gpu
dev = gpu_util.dev

# rows for each form: 1 decode (one block and runs of blocks), 2 tiles that quantize, 16, and the tiles
CASES = [(1, 1, 256), (1, 3, 512), (1, 17, 1024), (1, 129, 2048), (1, 31, 4096), (3, 257, 8192), (20, 33, 512),
         (32, 401, 4096), (5, 30001, 512), (16, 13003, 2048), (3, 4203, 8192), (20, 4401, 1024), (32, 4111, 4096),
         (300, 1, 256), (300, 127, 512), (300, 129, 768), (257, 255, 1024), (513, 257, 512), (300, 385, 512)]


def run(M, N, K, form, behind):
    codes, s = oracle.quantize_mxfp4(np.zeros((N, K)))
    pw = api.prepare_weight_fp4(torch.from_numpy(oracle.pack_fp4(codes)).to(dev()), torch.from_numpy(s).to(dev()))
    g = torch.Generator().manual_seed(N)
    x = synth.randn_bf16((M, K), 1.0, g).to(dev())
    around = torch.full((N + 5,), behind, dtype=torch.bfloat16)
    around[:N] = synth.randn_bf16((N,), 1.0, g)
    bias = around.to(dev())[:N]
    with ref.forced(form):
        y = api.linear_w4a4(x, pw, bias)
    torch.cuda.synchronize()
    off = (y != bias).nonzero()
    assert off.numel() == 0, (off.shape[0], off[0].tolist())


@pytest.mark.parametrize("form", [0, 1, 2, 16, 64, 128, 256])
@pytest.mark.parametrize("M,N,K", CASES)
def test_forms(form, M, N, K):
    run(M, N, K, form, float("nan"))


@pytest.mark.parametrize("form", [2, 64, 128, 256])
@pytest.mark.parametrize("K", [256, 512, 768])
def test_many_tiles_per_workgroup(form, K):
    run(*((2304, 8197) if form == 256 else (1500, 6501)), K, form, float("inf"))
