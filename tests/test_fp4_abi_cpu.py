"""Refusals of the MXFP4 x MXFP4 layer, of the sort by expert and of the
experts' products, without a GPU."""

import os

import pytest
import torch

from mxfp8_block_scaled_amd import api
from tests.test_abi_cpu import P
from tests.test_b128_abi_cpu import ALIGN, LD, NULLPTR, OK, SHAPE, WORKSPACE, refuse

pytestmark = pytest.mark.skipif(not os.path.exists(api.lib_path()), reason="libmxfp8.so not built")

BIG = 1 << 40


def test_quantize_act_packed_fp4():
    refuse(api.lib().mxfp8_quantize_act_packed_fp4, (P, 4, 512, 512, P, P, None), [
        (1, -1, SHAPE), (1, 0, OK), (1, (1 << 30) + 1, SHAPE), (2, 128, SHAPE), (2, 0, SHAPE), (2, (1 << 24) + 256, SHAPE),
        (0, None, NULLPTR), (4, None, NULLPTR), (5, None, NULLPTR), (3, 504, LD), (3, 516, LD), (0, P + 8, ALIGN),
        (4, P + 128, ALIGN), (5, P + 16, ALIGN)])
    assert api.lib().mxfp8_quantize_act_packed_fp4(P, 1 << 30, 1 << 24, 1 << 24, P, P, None) == SHAPE


def test_products():
    refuse(api.lib().mxfp8_gemm_packed_fp4, (P, P, 20, 512, P, P, 130, P, P, 130, None), [
        (2, -1, SHAPE), (2, 0, OK), (3, 128, SHAPE), (6, 0, SHAPE), (6, (1 << 24) + 1, SHAPE), (0, None, NULLPTR),
        (1, None, NULLPTR), (4, None, NULLPTR), (5, None, NULLPTR), (8, None, NULLPTR), (9, 129, LD), (0, P + 128, ALIGN),
        (4, P + 16, ALIGN), (7, P + 2, ALIGN), (8, P + 1, ALIGN)])
    refuse(api.lib().mxfp8_linear_w4a4, (P, 400, 4096, 4096, P, P, 130, P, P, 130, P, BIG, None), [
        (1, -1, SHAPE), (1, 0, OK), (2, 128, SHAPE), (6, 0, SHAPE), (0, None, NULLPTR), (4, None, NULLPTR),
        (5, None, NULLPTR), (8, None, NULLPTR), (3, 4088, LD), (3, 4097, LD), (9, 129, LD), (0, P + 8, ALIGN),
        (4, P + 16, ALIGN), (5, P + 16, ALIGN), (7, P + 2, ALIGN), (10, None, WORKSPACE), (11, 100, WORKSPACE),
        (10, P + 16, ALIGN)])
    # few rows need no workspace
    refuse(api.lib().mxfp8_linear_w4a4, (P, 4, 512, 512, P, P, 130, None, P, 130, None, 0, None), [(0, None, NULLPTR)])
    assert api.mxfp8_linear_w4a4_workspace_bytes(4, 130, 512) == 0
    assert api.mxfp8_linear_w4a4_workspace_bytes(4, 130, 16384) == 128 * 8192 + 128 * 512
    assert api.mxfp8_linear_w4a4_workspace_bytes(0, 130, 512) == 0
    with pytest.raises(api.MXFP8Error):
        api.mxfp8_linear_w4a4_workspace_bytes(4, 130, 384)
    assert api.lib().mxfp8_linear_w4a4(P, 1 << 30, 256, 256, P, P, 1 << 24, None, P, 1 << 24, P, BIG, None) == SHAPE
    assert api.mxfp8_debug_force_w4a4(7) == SHAPE


def test_sort():
    refuse(api.lib().mxfp8_moe_sort, (P, 4, 100, 8, P, P, P, None, 0, None), [
        (1, 2, SHAPE), (2, -1, SHAPE), (2, (1 << 26) + 1, SHAPE), (3, 0, SHAPE), (3, 257, SHAPE), (0, None, NULLPTR),
        (4, None, NULLPTR), (5, None, NULLPTR), (6, None, NULLPTR), (0, P + 2, ALIGN), (4, P + 2, ALIGN), (6, P + 1, ALIGN),
        (7, P + 16, ALIGN), (2, 5000, WORKSPACE)])
    refuse(api.lib().mxfp8_moe_sort, (P, 8, 5000, 8, P, P, P, P, BIG, None), [
        (0, P + 4, ALIGN), (7, None, WORKSPACE), (8, 16, WORKSPACE)])


def test_rows():
    refuse(api.lib().mxfp8_moe_permute, (P, 1, 10, 30, 30, 2, P, P, P, 30, None), [
        (1, 2, SHAPE), (2, -1, SHAPE), (2, 0, OK), (2, (1 << 24) + 1, SHAPE), (3, 0, SHAPE), (3, (1 << 24) + 1, SHAPE),
        (5, 0, SHAPE), (5, 17, SHAPE), (0, None, NULLPTR), (6, None, NULLPTR), (7, None, NULLPTR), (8, None, NULLPTR),
        (4, 29, LD), (9, 29, LD), (0, P + 1, ALIGN), (8, P + 1, ALIGN), (6, P + 2, ALIGN), (7, P + 2, ALIGN)])
    refuse(api.lib().mxfp8_moe_unpermute, (P, 0, 10, 30, 30, 2, P, P, P, P, 30, None), [
        (2, 0, OK), (5, 17, SHAPE), (0, None, NULLPTR), (9, None, NULLPTR), (4, 29, LD), (10, 29, LD), (0, P + 2, ALIGN),
        (8, P + 2, ALIGN), (9, P + 2, ALIGN)])
    refuse(api.lib().mxfp8_moe_unpermute_backward, (P, 0, 10, 30, 30, 2, P, P, P, 30, P, P, 30, P, None), [
        (2, 0, OK), (0, None, NULLPTR), (8, None, NULLPTR), (4, 29, LD), (9, 29, LD), (12, 29, LD), (11, P + 2, ALIGN),
        (13, P + 2, ALIGN)])
    assert api.lib().mxfp8_moe_unpermute_backward(P, 0, 10, 30, 30, 2, P, P, P, 30, P, None, 30, None, None) == NULLPTR
    assert api.lib().mxfp8_moe_permute(P, 0, 1 << 24, 1 << 24, 1 << 24, 1, P, P, P, 1 << 24, None) == SHAPE


def test_experts():
    refuse(api.lib().mxfp8_moe_prepare_experts_fp4, (P, P, 4, 130, 512, P, P, None), [
        (2, 0, SHAPE), (2, 257, SHAPE), (3, 0, SHAPE), (4, 128, SHAPE), (0, None, NULLPTR), (1, None, NULLPTR),
        (5, None, NULLPTR), (6, None, NULLPTR), (0, P + 8, ALIGN), (5, P + 16, ALIGN), (6, P + 16, ALIGN)])
    ok = (P, 6000, 512, 512, P, 4, P, 24000, 8, P, P, 130, P, 130, P, BIG, None)
    refuse(api.lib().mxfp8_moe_linear_w4a4, ok, [
        (1, 5999, SHAPE), (1, -1, SHAPE), (2, 128, SHAPE), (5, 0, SHAPE), (5, 17, SHAPE), (7, 24001, SHAPE), (8, 0, SHAPE),
        (8, 257, SHAPE), (11, 0, SHAPE), (0, None, NULLPTR), (6, None, NULLPTR), (9, None, NULLPTR), (10, None, NULLPTR),
        (12, None, NULLPTR), (3, 504, LD), (3, 514, LD), (13, 129, LD), (0, P + 8, ALIGN), (4, P + 2, ALIGN),
        (6, P + 2, ALIGN), (9, P + 16, ALIGN), (14, None, WORKSPACE), (15, 100, WORKSPACE), (14, P + 16, ALIGN),
        (4, None, SHAPE)])   # without the slots x has a row for each of them
    assert api.lib().mxfp8_moe_linear_w4a4(P, 0, 512, 512, None, 1, P, 0, 8, P, P, 130, P, 130, None, 0, None) == OK
    assert api.lib().mxfp8_moe_linear_w4a4(P, 1 << 26, 256, 256, None, 1, P, 1 << 26, 8, P, P, 130, P, 130, P, BIG,
                                           None) == SHAPE   # 2^33 bytes of quantized rows


def test_python_refusals():
    """What the wrappers refuse before the library is asked, on CPU tensors."""
    with pytest.raises(ValueError):
        api.moe_sort(torch.zeros(4, 2), 3)
    with pytest.raises(ValueError):
        api.moe_sort(torch.zeros(4, 2, dtype=torch.int32), 3)
    with pytest.raises(ValueError):
        api.moe_sort(torch.zeros(4, dtype=torch.int32), 3)
    order = api.MoEOrder(torch.zeros(4, 2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32),
                         torch.zeros(4, dtype=torch.int32))
    for bad in (torch.zeros(4, 8, dtype=torch.float16), torch.zeros(3, 8), torch.zeros(8), torch.zeros(4, 8)):
        with pytest.raises(ValueError):
            api.moe_permute(bad, order)
    with pytest.raises(ValueError):
        api.moe_unpermute(torch.zeros(4, 8), order)
    with pytest.raises(ValueError):
        api.moe_permute(torch.zeros(4, 8), None)
    with pytest.raises(ValueError):
        api.linear_w4a4(torch.zeros(4, 256, dtype=torch.bfloat16), object())
    with pytest.raises(ValueError):
        api.moe_linear_w4a4(torch.zeros(4, 256, dtype=torch.bfloat16), object(), order)
    with pytest.raises(ValueError):
        api.quantize_act_packed_fp4(torch.zeros(4, 256))


def test_launches_of_more_than_32_bits():
    """Refused, not wrapped: a launch has fewer than 2^32 threads."""
    lib = api.lib()
    assert lib.mxfp8_moe_permute(P, 1, 1 << 24, 2048, 2048, 1, P, P, P, 2048, None) == SHAPE
    assert lib.mxfp8_moe_unpermute(P, 1, 1 << 24, 2048, 2048, 1, P, P, None, P, 2048, None) == SHAPE
    assert lib.mxfp8_quantize_act_packed_fp4(P, 1 << 28, 512, 512, P, P, None) == SHAPE
    assert lib.mxfp8_moe_prepare_experts_fp4(P, P, 1, 1 << 24, 8192, P, P, None) == SHAPE
    # one below each: past the shape checks
    assert lib.mxfp8_moe_permute(None, 1, (1 << 24) - 1, 2048, 2048, 1, P, P, P, 2048, None) == NULLPTR
    assert lib.mxfp8_quantize_act_packed_fp4(None, (1 << 28) - 128, 512, 512, P, P, None) == NULLPTR
