"""128-block operands given to an entry point of the MX format: refused before
anything is read (the MX kernels would read past the shorter scales)."""

import pytest
import torch

from mxfp8_block_scaled_amd import api


def test_gemm_prequant_refuses_a_128_block_weight():
    pw = api.PreparedWeightB128(torch.empty(128 * 256, dtype=torch.uint8), torch.empty(2), 128, 256)
    q, s = torch.empty(4, 256, dtype=torch.uint8), torch.empty(4, 8, dtype=torch.uint8)
    with pytest.raises(ValueError, match="128-blocks"):
        api.gemm_prequant(q, s, pw)


def test_gemm_packed_refuses_mixed_blocks():
    pw = api.PreparedWeightB128(torch.empty(128 * 256, dtype=torch.uint8), torch.empty(2), 128, 256)
    mx = api.PreparedWeight(torch.empty(128 * 256, dtype=torch.uint8), torch.empty(128 * 8, dtype=torch.uint8), 128, 256)
    q, s = torch.empty(128 * 256, dtype=torch.uint8), torch.empty(128 * 8, dtype=torch.uint8)
    for pa, w in ((api.PackedActivation(q, s, 4, 256), pw), (api.PackedActivation(q, s, 4, 256, block=128), mx)):
        with pytest.raises(ValueError, match="scale per"):
            api.gemm_packed(pa, w)
