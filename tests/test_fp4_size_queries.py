"""The size queries of the MXFP4 entry points refuse what the calls refuse, without a GPU; and the sort's workspace."""

import ctypes
import os

import pytest

from mxfp8_block_scaled_amd import api
from tests.test_abi_cpu import P
from tests.test_b128_abi_cpu import NULLPTR, OK, SHAPE

pytestmark = pytest.mark.skipif(not os.path.exists(api.lib_path()), reason="libmxfp8.so not built")

BIG = 1 << 62


def query(name, *sizes, outs=1):
    out = [ctypes.c_size_t(0) for _ in range(outs)]
    st = getattr(api.lib(), name)(*sizes, *[ctypes.byref(o) for o in out])
    return st, tuple(o.value for o in out)


# rows x columns in tiles of 64 x 128 from 2^30 on, and threads of the quantizer from 2^32 on
DENSE = [((1 << 30, 1 << 24, 256), SHAPE), ((1 << 22, 1 << 21, 256), SHAPE), ((1 << 22, (1 << 21) - 128, 256), OK),
         ((1 << 28, 128, 512), SHAPE), (((1 << 28) - 128, 128, 512), OK), ((1 << 20, 128, 1 << 17), SHAPE),
         ((1, 1 << 24, 1 << 24), OK), ((0, 1 << 24, 1 << 24), OK)]


@pytest.mark.parametrize("shape,want", DENSE)
def test_linear(shape, want):
    M, N, K = shape
    assert query("mxfp8_linear_w4a4_workspace_bytes", M, N, K)[0] == want
    # (the call: refused for the shape, or else for what it lacks)
    st = api.lib().mxfp8_linear_w4a4(P, M, K, K, P, P, N, None, None, N, P, BIG, None)
    assert st == (OK if M == 0 else NULLPTR)
    if want == SHAPE:
        assert api.lib().mxfp8_linear_w4a4(P, M, K, K, P, P, N, None, P, N, P, BIG, None) == SHAPE


@pytest.mark.parametrize("M,K,want", [(1 << 28, 512, SHAPE), ((1 << 28) - 128, 512, OK), (1 << 30, 256, SHAPE),
                                      (1 << 20, 1 << 17, SHAPE), (128, 1 << 24, OK)])
def test_packed_activations(M, K, want):
    st, sizes = query("mxfp8_packed_act_fp4_bytes", M, K, outs=2)
    assert st == want
    call = api.lib().mxfp8_quantize_act_packed_fp4
    if want == SHAPE:
        assert call(P, M, K, K, P, P, None) == SHAPE
    else:
        assert sizes == (M * K // 2, M * K // 32) and call(None, M, K, K, P, P, None) == NULLPTR


@pytest.mark.parametrize("E,N,K,want", [(1, 1 << 24, 8192, SHAPE), (256, 1 << 24, 8192, SHAPE), (1, 1 << 24, 7936, OK),
                                        (2, (1 << 24) - 1, 8192, SHAPE), (256, 1 << 20, 8192, OK), (4, 130, 512, OK)])
def test_experts_weights(E, N, K, want):
    st, sizes = query("mxfp8_moe_prepared_experts_fp4_bytes", E, N, K, outs=2)
    assert st == want
    if want == SHAPE:
        assert api.lib().mxfp8_moe_prepare_experts_fp4(P, P, E, N, K, P, P, None) == SHAPE
    else:
        pad = (N + 127) // 128 * 128
        assert sizes == (E * pad * K // 2, E * pad * K // 32)


@pytest.mark.parametrize("R,N,want", [(1 << 26, 1 << 17, SHAPE), (1 << 26, (1 << 17) - 128, OK), ((1 << 26) + 1, 128, SHAPE)])
def test_experts(R, N, want):
    """64-row tiles of the rows and one more for each expert, by 128 columns, below 2^30."""
    K, E = 256, 256
    x_rows = R // 16
    assert query("mxfp8_moe_linear_w4a4_workspace_bytes", x_rows, R, N, K, E)[0] == want
    st = api.lib().mxfp8_moe_linear_w4a4(P, x_rows, K, K, P, 16, P, R, E, P, P, N, None, N, P, BIG, None)
    assert st == (SHAPE if want == SHAPE else NULLPTR)


def test_sort_workspace():
    """One count for each expert and for none of them, of each workgroup: chunks of 1024 slots or more, 256 workgroups at
    most; none for up to 4096 slots, which one workgroup sorts."""
    for slots in (0, 1, 1024, 4096, 4097, 5000, 5121, 1 << 17, (1 << 18) - 1, 1 << 18, (1 << 18) + 1, 300001, 1 << 26):
        chunk = max(1024, -(-slots // 256))
        n = -(-slots // chunk) if slots > 4096 else 0
        for E in (1, 8, 256):
            assert query("mxfp8_moe_sort_workspace_bytes", slots, E) == (OK, (n * (E + 1) * 4,))
