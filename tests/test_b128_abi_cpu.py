"""Refusals of the 128-block, weight-gradient and balance-loss entry points,
without a GPU: every invalid argument is rejected before a device is touched;
the Python wrappers refuse what the library could not check."""

import os

import numpy as np
import pytest
import torch

from mxfp8_block_scaled_amd import api
from tests import b128_ref as ref
from tests.test_abi_cpu import GPU_VISIBLE, P, expect_no_device

pytestmark = pytest.mark.skipif(not os.path.exists(api.lib_path()), reason="libmxfp8.so not built")

OK, NULLPTR, SHAPE, ALIGN, LD, WORKSPACE = 0, -1, -2, -3, -4, -5


def refuse(fn, ok, cases):
    """Each case: (argument index, bad value, status)."""
    expect_no_device(fn, *ok)
    for at, value, status in cases:
        args = list(ok)
        args[at] = value
        assert fn(*args) == status, (at, value, status, fn(*args))


def test_quantize_b128():
    refuse(api.lib().mxfp8_quantize_b128, (P, 4, 144, 144, P, 144, P, 2, None), [
        (1, -1, SHAPE), (1, 0, OK), (1, (1 << 30) + 1, SHAPE), (2, 136, SHAPE), (2, 0, SHAPE), (2, (1 << 24) + 16, SHAPE),
        (0, None, NULLPTR), (4, None, NULLPTR), (6, None, NULLPTR), (3, 136, LD), (3, 148, LD), (5, 128, LD), (5, 152, LD),
        (7, 1, LD), (0, P + 8, ALIGN), (4, P + 8, ALIGN)])


def test_quantize_act_packed_b128():
    refuse(api.lib().mxfp8_quantize_act_packed_b128, (P, 4, 144, 144, P, P, None), [
        (1, -1, SHAPE), (1, 0, OK), (2, 100, SHAPE), (0, None, NULLPTR), (4, None, NULLPTR), (5, None, NULLPTR),
        (3, 128, LD), (3, 150, LD), (0, P + 2, ALIGN), (4, P + 128, ALIGN), (5, P + 16, ALIGN)])
    refuse(api.lib().mxfp8_dequantize_act_packed, (P, P, 4, 144, P, 144, None), [
        (2, -1, SHAPE), (2, 0, OK), (3, 100, SHAPE), (0, None, NULLPTR), (1, None, NULLPTR), (4, None, NULLPTR),
        (5, 128, LD), (5, 150, LD), (0, P + 16, ALIGN), (1, P + 16, ALIGN), (4, P + 8, ALIGN)])
    # sizes whose launch would leave 32-bit grids
    assert api.lib().mxfp8_quantize_act_packed_b128(P, 1 << 30, 1 << 24, 1 << 24, P, P, None) == SHAPE


def test_weight_b128():
    refuse(api.lib().mxfp8_prepare_weight_b128, (P, P, 130, 144, 144, 2, 0, P, P, None), [
        (2, 0, SHAPE), (3, 100, SHAPE), (6, 1, SHAPE), (0, None, NULLPTR), (1, None, NULLPTR), (7, None, NULLPTR),
        (8, None, NULLPTR), (4, 128, LD), (4, 152, LD), (5, 1, LD), (0, P + 8, ALIGN), (1, P + 2, ALIGN), (7, P + 16, ALIGN),
        (8, P + 16, ALIGN)])
    expect_no_device(api.lib().mxfp8_prepare_weight_b128, P, P, 144, 144, 144, 2, 1, P, P, None)
    refuse(api.lib().mxfp8_quantize_weight_b128, (P, 144, 144, 144, P, 144, P, 2, P, P, P, P, None), [
        (1, 130, SHAPE), (2, 100, SHAPE), (0, None, NULLPTR), (4, None, NULLPTR), (6, None, NULLPTR), (8, None, NULLPTR),
        (9, None, NULLPTR), (10, None, NULLPTR), (11, None, NULLPTR), (3, 128, LD), (3, 148, LD), (5, 152, LD), (7, 1, LD),
        (0, P + 8, ALIGN), (4, P + 8, ALIGN), (8, P + 64, ALIGN), (11, P + 64, ALIGN)])
    # no output wanted at all
    assert api.lib().mxfp8_quantize_weight_b128(P, 144, 144, 144, None, 0, None, 0, None, None, None, None, None) == NULLPTR
    # a weight that is not transposed takes any N
    expect_no_device(api.lib().mxfp8_quantize_weight_b128, P, 131, 144, 144, P, 144, P, 2, P, P, None, None, None)
    assert api.mxfp8_prepared_weight_b128_bytes(130, 144) == (256 * 256, 16)
    for bad in ((0, 128), (5, 8), (5, 24)):
        with pytest.raises(api.MXFP8Error):
            api.mxfp8_prepared_weight_b128_bytes(*bad)


@pytest.mark.parametrize("M", [4, 300])
def test_linear_b128(M):
    N, K = 130, 272
    ws = api.mxfp8_linear_b128_workspace_bytes(M, N, K)
    assert ws == 0 if M <= 16 else ws >= 384 * 384
    refuse(api.mxfp8_linear_b128, (P, M, K, K, P, P, N, None, P, N, P, ws, None), [
        (1, -1, SHAPE), (1, 0, OK), (2, 264, SHAPE), (6, 0, SHAPE), (0, None, NULLPTR), (4, None, NULLPTR),
        (5, None, NULLPTR), (8, None, NULLPTR), (3, 264, LD), (3, 276, LD), (9, 129, LD), (10, P + 64, ALIGN),
        (0, P + 8, ALIGN), (4, P + 64, ALIGN), (5, P + 64, ALIGN), (7, P + 1, ALIGN), (8, P + 1, ALIGN)])
    if ws:
        refuse(api.mxfp8_linear_b128, (P, M, K, K, P, P, N, None, P, N, P, ws, None), [
            (10, None, WORKSPACE), (11, ws - 1, WORKSPACE)])
    else:                                          # decode: no workspace
        expect_no_device(api.mxfp8_linear_b128, P, M, K, K, P, P, N, None, P, N, None, 0, None)
    need = api._bytes("mxfp8_gemm_packed_b128_workspace_bytes", M, N, K)
    refuse(api.lib().mxfp8_gemm_packed_b128, (P, P, M, K, P, P, N, None, P, N, P, need, None), [
        (2, -1, SHAPE), (2, 0, OK), (3, 264, SHAPE), (6, 0, SHAPE), (0, None, NULLPTR), (1, None, NULLPTR),
        (8, None, NULLPTR), (9, 129, LD), (10, None, WORKSPACE), (11, need - 1, WORKSPACE), (0, P + 64, ALIGN),
        (1, P + 64, ALIGN)])


@pytest.mark.parametrize("M,N,K", [(33, 1, 16), (40, 515, 272), (1000, 4096, 4096), (64, 128, 65536), (8192, 28672, 8192)])
def test_split_workspace_holds_the_partials(M, N, K):
    """The GEMM's workspace is its activations and its fp32 partials."""
    act = -(-M // 128) * 128 * (-(-K // 128) * 128)
    part = api._bytes("mxfp8_gemm_packed_b128_workspace_bytes", M, N, K)
    total = api.mxfp8_linear_b128_workspace_bytes(M, N, K)
    row = M * (-(-N // 4) * 4) * 4
    up = lambda v: -(-v // 256) * 256
    splits = 0 if part == 256 and up(2 * row) > 256 else part // row
    assert splits in (0, 2, 4, 8) or part == 256
    assert total >= act + act // 32 + (part if splits else 0)


def test_wgrad():
    M, N, K = 100, 136, 272
    fn = api.lib().mxfp8_linear_wgrad
    need = api._bytes("mxfp8_linear_wgrad_workspace_bytes", M, N, K)
    ok = (P, M, N, N, P, P, K, P, 0, K, P, 0, 0, P, need, None)
    refuse(fn, ok, [
        (1, -1, SHAPE), (2, 0, SHAPE), (2, 132, SHAPE), (6, 264, SHAPE), (8, 2, SHAPE), (0, None, NULLPTR),
        (4, None, NULLPTR), (5, None, NULLPTR), (7, None, NULLPTR), (3, 128, LD), (3, 140, LD), (3, (1 << 24) + 8, LD),
        (9, 264, LD), (9, 276, LD), (0, P + 8, ALIGN), (7, P + 8, ALIGN), (10, P + 2, ALIGN), (4, P + 16, ALIGN),
        (5, P + 16, ALIGN), (11, 2, SHAPE), (13, P + 16, ALIGN)])
    many = api._bytes("mxfp8_linear_wgrad_workspace_bytes", 5000, N, K)   # tiles in several runs: partial sums
    assert many > 0
    refuse(fn, ok[:1] + (5000,) + ok[2:14] + (many, None), [(13, None, WORKSPACE), (14, many - 1, WORKSPACE)])
    for at in (8, 11):                             # accumulation is fp32
        bf16 = list(ok)
        bf16[at], bf16[12] = 1, 1
        assert fn(*bf16) == SHAPE
    empty = list(ok)
    empty[0] = empty[4] = empty[5] = None          # no tokens: no operands
    empty[1], empty[3] = 0, 0
    expect_no_device(fn, *empty)


@pytest.mark.parametrize("keep", [0, 1, 2, 3])
@pytest.mark.parametrize("M", [4, 100])
def test_training_step(keep, M):
    N, K = 144, 272
    kept, fws, bws = api._layer_bytes(M, N, K, keep)
    assert (kept > 0) == (keep > 0)
    fwd, bwd = api.lib().mxfp8_linear_b128_forward, api.lib().mxfp8_linear_b128_backward
    refuse(fwd, (P, M, K, K, P, N, K, P, P, N, keep, P, P, fws, None), [
        (1, -1, SHAPE), (2, 264, SHAPE), (5, 136, SHAPE), (10, 4, SHAPE), (0, None, NULLPTR), (4, None, NULLPTR),
        (8, None, NULLPTR), (3, 264, LD), (3, 276, LD), (6, 264, LD), (9, 143, LD), (0, P + 8, ALIGN), (4, P + 8, ALIGN),
        (7, P + 1, ALIGN), (11, P + 16, ALIGN), (12, None, WORKSPACE), (13, fws - 1, WORKSPACE), (12, P + 16, ALIGN)])
    dx, dw = (P if keep & 1 else None), (P if keep & 2 else None)
    ok = (P, M, N, N, K, keep, P, dx, K, dw, 1, K, dw, 1, P, bws, None)
    cases = [(1, -1, SHAPE), (2, 136, SHAPE), (4, 264, SHAPE), (5, 4, SHAPE), (6, P + 16, ALIGN)]
    if keep:
        cases += [(0, None, NULLPTR), (3, 136, LD), (3, 146, LD), (0, P + 8, ALIGN), (6, None, NULLPTR)]
        assert fwd(P, M, K, K, P, N, K, P, P, N, keep, None, P, fws, None) == NULLPTR
    if bws:
        cases += [(14, None, WORKSPACE), (15, bws - 1, WORKSPACE), (14, P + 16, ALIGN)]
    if keep & 1:
        cases += [(8, 271, LD), (7, P + 1, ALIGN)]
    else:
        cases += [(7, P, SHAPE)]                   # its operand was not kept
    if keep & 2:
        cases += [(10, 2, SHAPE), (11, 264, LD), (9, P + 8, ALIGN), (13, 2, SHAPE), (9, None, SHAPE)]
    else:
        cases += [(9, P, SHAPE), (12, P, SHAPE)]
    if keep:
        refuse(bwd, ok, cases)
    else:
        for at, value, status in cases:
            args = list(ok)
            args[at] = value
            assert bwd(*args) == status


def test_balance():
    lib = api.lib()
    need = api._bytes("mxfp8_moe_balance_workspace_bytes", 50, 24)
    refuse(lib.mxfp8_moe_balance, (P, 0, 50, 24, 24, 4, None, 0.1, 0.0, P, P, P, P, need, None), [
        (1, 2, SHAPE), (2, -1, SHAPE), (2, 1 << 31, SHAPE), (3, 0, SHAPE), (3, 257, SHAPE), (5, 0, SHAPE), (5, 17, SHAPE),
        (5, 25, SHAPE), (0, None, NULLPTR), (9, None, NULLPTR), (10, None, NULLPTR), (11, None, NULLPTR), (4, 23, LD),
        (0, P + 2, ALIGN), (9, P + 2, ALIGN), (12, None, WORKSPACE), (13, need - 1, WORKSPACE), (12, P + 16, ALIGN)])
    refuse(lib.mxfp8_moe_balance_backward, (P, 1, 50, 24, 24, 4, None, 0.1, 0.0, P, P, None, P, 24, None), [
        (1, -1, SHAPE), (2, -1, SHAPE), (2, 0, OK), (3, 257, SHAPE), (5, 25, SHAPE), (0, None, NULLPTR), (9, None, NULLPTR),
        (10, None, NULLPTR), (12, None, NULLPTR), (4, 23, LD), (13, 23, LD), (0, P + 1, ALIGN), (12, P + 1, ALIGN),
        (11, P + 2, ALIGN)])


def test_wrappers_refuse():
    """What would reach the library as a wrong pointer or size is refused in
    Python: CPU tensors, wrong types, shapes that do not fit."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for fn in (api.quantize_act_b128, api.quantize_act_packed_b128, api.quantize_weight_b128, api.prepare_weight_b128_bf16):
        with pytest.raises(ValueError, match="GPU"):
            fn(x)
        with pytest.raises(ValueError, match="bfloat16"):
            fn(x.float())
    with pytest.raises(ValueError, match="GPU"):
        api.linear_b128(x, x)
    with pytest.raises(ValueError, match="bfloat16"):
        api.linear_b128(x.half(), x)
    with pytest.raises(ValueError, match="GPU"):
        api.moe_balance(torch.zeros(3, 4), 1)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        api.moe_balance(torch.zeros(3, 4, dtype=torch.float16), 1)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        api.moe_balance_loss(torch.zeros(4), 1)
    with pytest.raises(ValueError, match="GPU"):
        api.prepare_weight_b128(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 1))


@pytest.mark.gpu
def test_wrappers_refuse_on_the_gpu():
    d = torch.device("cuda", 0)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=d)
    w = torch.zeros(32, 64, dtype=torch.uint8, device=d)
    pw = api.prepare_weight_b128(w, torch.ones(1, 1, device=d))
    pa, mx = api.quantize_act_packed_b128(x), api.quantize_act_packed(torch.zeros(4, 256, dtype=torch.bfloat16, device=d))
    dy = torch.zeros(4, 32, dtype=torch.bfloat16, device=d)
    f32 = lambda *s: torch.zeros(*s, device=d)
    cases = [
        lambda: api.prepare_weight_b128(w, torch.ones(1, 1, dtype=torch.float64, device=d)),
        lambda: api.prepare_weight_b128(torch.zeros(200, 64, dtype=torch.uint8, device=d), torch.ones(1, 1, device=d)),
        lambda: api.prepare_weight_b128(w, torch.ones(1, 1)),
        lambda: api.linear(x[:, :48], pw),
        lambda: api.linear(x.float(), pw),
        lambda: api.linear(x, pw, bias=torch.zeros(31, dtype=torch.bfloat16, device=d)),
        lambda: api.linear(x, pw, bias=torch.zeros(32, dtype=torch.bfloat16)),
        lambda: api.linear(x, pw, out=f32(4, 32)),
        lambda: api.linear(x, pw, out=torch.zeros(3, 32, dtype=torch.bfloat16, device=d)),
        lambda: api.linear(x, pw, out=torch.zeros(32, 4, dtype=torch.bfloat16, device=d).t()),
        lambda: api.gemm_packed(mx, api.PreparedWeightB128(pw.w_packed, pw.s_packed, 32, 256)),
        lambda: api.gemm_packed(pa, api.PreparedWeight(pw.w_packed, pw.s_packed, 32, 64)),
        lambda: api.linear_wgrad(dy[:3], pa),
        lambda: api.linear_wgrad(dy, pa, accumulate=True),
        lambda: api.linear_wgrad(dy, pa, out=f32(32, 64), bias_grad=True, accumulate=True),
        lambda: api.linear_wgrad(dy, pa, out=f32(32, 48)),
        lambda: api.linear_wgrad(dy, pa, out=f32(64, 32).t()),
        lambda: api.linear_wgrad(dy, pa, out=torch.zeros(32, 64, device=d, dtype=torch.bfloat16), accumulate=True),
        lambda: api.linear_wgrad(dy, pa, dtype=torch.float16),
        lambda: api.linear_wgrad(dy, pa, bias_grad=True, out_bias=f32(64)[::2]),
        lambda: api.linear_wgrad(dy.float(), pa),
        lambda: api.linear_b128(x, torch.zeros(24, 64, dtype=torch.bfloat16, device=d)),
        lambda: api.linear_b128(x, torch.zeros(32, 48, dtype=torch.bfloat16, device=d)),
        lambda: api.moe_balance(f32(3, 4), 1, valid=torch.ones(4, dtype=torch.bool, device=d)),
        lambda: api.moe_balance(f32(3, 4), 1, valid=f32(3)),
        lambda: api.moe_balance(f32(3, 4), 1, valid=torch.ones(3, dtype=torch.bool)),
        lambda: api.moe_balance_backward(f32(3, 4), 1, f32(4), torch.ones(1, dtype=torch.int32, device=d)),
        lambda: api.moe_balance_backward(f32(3, 4), 1, torch.ones(3, dtype=torch.int32, device=d),
                                         torch.ones(1, dtype=torch.int32, device=d)),
    ]
    for i, case in enumerate(cases):
        with pytest.raises(ValueError):
            case()
            pytest.fail(f"case {i} was taken")
    for bad in (lambda: api.moe_balance(f32(3, 300), 1), lambda: api.moe_balance(f32(3, 4), 5),
                lambda: api.linear_wgrad(torch.zeros(4, 12, dtype=torch.bfloat16, device=d), pa),
                lambda: api.quantize_act_b128(torch.zeros(4, 40, dtype=torch.bfloat16, device=d))):
        with pytest.raises(api.MXFP8Error):
            bad()


def test_reference_rules():
    """The 64-bit forms the GPU tests compare with, against torch's cast and by
    hand."""
    v = np.concatenate([np.linspace(-448, 448, 20001), np.exp2(np.linspace(-12, 8, 4001))])
    want = torch.from_numpy(v).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3_round(v.astype(np.float32)), want)
    amax = [0.0, 448.0, 449.0, 448.0 * 2 ** -20, 1.0, 1.75, 1.76, 2.0 ** -133, float("inf"), float("nan")]
    assert ref.scale_bytes(amax).tolist() == [0, 127, 128, 107, 119, 119, 120, 0, 255, 255]
    x = np.zeros((2, 200))
    x[0, 3], x[1, 150] = 3.0, -500.0
    q, s, d = ref.quantize(x)
    assert s.tolist() == [[120, 0], [0, 128]] and q[0, 3] == 384.0 and q[1, 150] == -256.0 and d[1, 150] == -512.0
