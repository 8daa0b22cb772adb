"""MXFP4 operands given to an entry point that reads 8-bit ones, and experts' weights to one that takes a single weight:
refused before anything is read (the kernels would read past the shorter codes)."""

import pytest
import torch

from mxfp8_block_scaled_amd import api

M, N, K = 4, 128, 256


def bytes_(*shape):
    return torch.empty(*shape, dtype=torch.uint8)


X = torch.empty(M, K, dtype=torch.bfloat16)
ACT8 = api.PackedActivation(bytes_(128 * K), bytes_(128 * K // 32), M, K)
ACT4 = api.PackedActivationFP4(bytes_(128 * K // 2), bytes_(128 * K // 32), M, K)
W8 = api.PreparedWeight(bytes_(N * K), bytes_(N * K // 32), N, K)
W4 = api.PreparedWeightFP4(bytes_(N * K // 2), bytes_(N * K // 32), N, K)
EXPERTS = api.ExpertWeightsFP4(bytes_(N * K // 2), bytes_(N * K // 32), 1, N, K)


class Library:
    def __getattr__(self, name):
        raise AssertionError(f"{name} was reached")


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    monkeypatch.setattr(api, "lib", lambda: Library())
    monkeypatch.setattr(api, "_require_cuda", lambda t, name: None)


def test_weight_gradient_of_mxfp4_activations():
    dy = torch.empty(M, N, dtype=torch.bfloat16)
    for kw in ({}, {"bias_grad": True}, {"out": torch.empty(N, K)}):
        with pytest.raises(ValueError, match="MXFP4"):
            api.linear_wgrad(dy, ACT4, **kw)


def test_prequantized_activations_and_an_mxfp4_weight():
    for pw in (W4, EXPERTS):
        with pytest.raises(ValueError, match="MXFP8 weight"):
            api.gemm_prequant(bytes_(M, K), bytes_(M, K // 32), pw)


def test_packed_activations():
    for pa, pw in ((ACT4, W8), (ACT8, W4), (ACT8, EXPERTS), (ACT4, EXPERTS)):
        with pytest.raises(ValueError, match="MXFP4|weight"):
            api.gemm_packed(pa, pw)


def test_layers():
    for f in (api.linear, api.linear_w4a4):
        with pytest.raises(ValueError, match="weight"):
            f(X, EXPERTS)
    with pytest.raises(ValueError, match="MXFP4 weight"):
        api.linear_w4a4(X, W8)


def test_dequantize():
    with pytest.raises(NotImplementedError):
        ACT4.dequantize()
