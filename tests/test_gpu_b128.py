"""The FP8 linear layer with 128-blocks on the GPU: quantizers byte-exact,
layout and GEMM against 64-bit forms, over sizes that end inside blocks,
tiles and split runs; strides, views, streams, captured graphs."""

import numpy as np
import pytest
import torch

from mxfp8_block_scaled_amd import api
from tests import b128_ref as ref
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


def randn(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def spiky(M, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp(torch.randn(1, K, generator=g))
    x = torch.where(torch.rand(M, K, generator=g) < 0.01, x * 50, x)
    return x.to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def edge_rows():
    """Rows of two blocks: every exponent with the mantissas around the 448
    border, zeros, subnormals, infinities and NaN."""
    rows = []
    for f in list(range(0, 12)) + [126, 127, 128, 200, 253, 254]:
        for mant in (0, 1, 95, 96, 97, 127):
            v = (f << 7) | mant
            r = np.zeros(256, dtype=np.uint16)
            r[5] = v
            r[6] = v | 0x8000
            r[7] = v >> 1
            r[130] = max(v - 1, 0)
            r[255] = 0x8000
            rows.append(r)
    for bad in (0x7F80, 0xFF80, 0x7FC0, 0xFFFF):
        r = np.full(256, 0x3F80, dtype=np.uint16)
        r[200] = bad
        rows.append(r)
    return torch.from_numpy(np.stack(rows).view(np.int16)).view(torch.bfloat16)


def check_quantized(x, q, s):
    K = x.shape[1]
    with np.errstate(invalid="ignore", over="ignore"):
        want_q, want_s, _ = ref.quantize(f64(x))
    np.testing.assert_array_equal(s, want_s)
    bad = np.repeat(want_s == 255, 128, 1)[:, :K]
    got = ref.decode(q)
    assert np.array_equal(got[~bad], want_q[~bad])
    neg = np.signbit(got) == np.signbit(f64(x))
    assert neg[~bad].all()


@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (17, 272), (128, 256), (130, 1040), (5, 8208)])
def test_quantize_act(M, K):
    x = spiky(M, K, M + K)
    q, s = api.quantize_act_b128(x.to(dev()))
    check_quantized(x, q.cpu(), s.cpu().numpy())


def test_quantize_act_edges():
    x = edge_rows()
    q, s = api.quantize_act_b128(x.to(dev()))
    check_quantized(x, q.cpu(), s.cpu().numpy())


@pytest.mark.parametrize("M,K", [(1, 16), (3, 144), (16, 128), (129, 512), (300, 1040), (2100, 2048)])
def test_packed_quantizer_holds_the_same_values(M, K):
    x = spiky(M, K, 3 * M + K)
    pa = api.quantize_act_packed_b128(x.to(dev()))
    _, _, want = ref.quantize(f64(x))
    assert np.array_equal(f64(pa.dequantize()), want)
    if K % 256 == 0:   # the bytes, pad rows among them
        q, s = pa.unpack()
        rq, rs = api.quantize_act_b128(x.to(dev()))
        assert torch.equal(q[:M], rq) and torch.equal(s[:M], rs.repeat_interleave(4, 1))
        assert not q[M:].any() and not s[M:].any()


def test_dequantize_of_an_mx_checkpoint():
    x = spiky(70, 512, 5)
    pa = api.quantize_act_packed(x.to(dev()))
    q, s = pa.unpack()
    want = ref.decode(q.cpu())[:70] * np.exp2(np.repeat(s.cpu().numpy()[:70].astype(float), 32, 1) - 127)
    assert np.array_equal(f64(pa.dequantize()), want)


@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (130, 272), (256, 1040), (48, 96)])
def test_quantize_weight(N, K):
    w = spiky(N, K, N * K)
    q, s = api.quantize_weight_b128(w.to(dev()))
    want_q, want_s, _ = ref.quantize(f64(w), rows=128)
    assert np.array_equal(ref.decode(q.cpu()), want_q)
    assert np.array_equal(f64(s), np.exp2(want_s.astype(float) - 127))


@pytest.mark.parametrize("N,K", [(16, 16), (128, 256), (144, 272), (400, 1040)])
def test_prepared_forms_agree(N, K):
    """Both orientations in one pass = quantize, then prepare each."""
    w = spiky(N, K, N + K).to(dev())
    q, s = api.quantize_weight_b128(w)
    pw, pt = api.prepare_weight_b128_bf16(w)
    for got, want in ((pw, api.prepare_weight_b128(q, s)), (pt, api.prepare_weight_b128(q, s, transpose=True))):
        assert (got.N, got.K) == (want.N, want.K)
        assert torch.equal(got.w_packed, want.w_packed) and torch.equal(got.s_packed, want.s_packed)
    # the transposed form is the form of the transposed bytes
    tt = api.prepare_weight_b128(q.t().contiguous(), s.t().contiguous())
    assert torch.equal(tt.w_packed, pt.w_packed) and torch.equal(tt.s_packed, pt.s_packed)


def make_weight(N, K, seed):
    """E4M3 bytes with arbitrary fp32 block scales, as checkpoints hold them."""
    g = torch.Generator().manual_seed(seed)
    v = (torch.randn(N, K, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = torch.exp(torch.randn(-(-N // 128), -(-K // 128), generator=g)) * 1e-3
    return v.view(torch.uint8), s


def check_linear(x, wq, ws, bias, y):
    """y bf16 [M, N] against the 64-bit product of the quantized operands."""
    N, K = wq.shape
    _, _, A = ref.quantize(f64(x))
    W = ref.decode(wq) * ref.spread(ws.numpy(), N, K)
    want = A @ W.T + (0 if bias is None else f64(bias))
    err = np.abs(f64(y) - want)
    bound = 2.0 ** -8 * np.abs(want) + ref.gemm_bound(A, W)
    assert np.isfinite(f64(y)).all()
    assert (err <= bound).all(), (float((err / bound).max()), np.argwhere(err > bound)[:4])
    if want.size > 64:
        assert np.linalg.norm(err) <= 2.0 ** -8 * np.linalg.norm(want)


SIZES = [(1, 1, 16), (1, 130, 128), (2, 16, 144), (7, 130, 256), (16, 4000, 2064), (13, 512, 8336), (16, 64, 20000),
         (17, 128, 128), (17, 130, 1040), (33, 515, 272), (64, 256, 4096), (65, 300, 512), (128, 128, 16),
         (129, 257, 1152), (200, 4096, 640), (300, 1000, 2064), (513, 384, 4112), (1024, 2048, 1024), (1000, 4000, 400)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("with_bias", [False, True])
def test_linear(M, N, K, with_bias):
    x = spiky(M, K, M + N + K)
    wq, ws = make_weight(N, K, N + K)
    bias = randn((N,), 9) if with_bias else None
    pw = api.prepare_weight_b128(wq.to(dev()), ws.to(dev()))
    y = api.linear(x.to(dev()), pw, None if bias is None else bias.to(dev()))
    assert y.shape == (M, N)
    check_linear(x, wq, ws, bias, y)


@pytest.mark.parametrize("M,N,K", [(1, 130, 272), (40, 96, 640), (260, 513, 1040)])
def test_gemm_packed_is_the_tile_path(M, N, K):
    x = spiky(M, K, 1)
    wq, ws = make_weight(N, K, 2)
    pw = api.prepare_weight_b128(wq.to(dev()), ws.to(dev()))
    y = api.gemm_packed(api.quantize_act_packed_b128(x.to(dev())), pw)
    check_linear(x, wq, ws, None, y)
    if M > 16:
        assert torch.equal(y, api.linear(x.to(dev()), pw))


@pytest.mark.parametrize("M", [5, 150])
def test_one_hot_weight_places_every_element(M):
    """y = one element of x per output: layout and scale placement, exactly."""
    K, N = 1040, 1040
    x = spiky(M, K, 4)
    perm = torch.randperm(K, generator=torch.Generator().manual_seed(1))
    wq = torch.zeros(N, K)
    wq[torch.arange(N), perm] = 1.0
    ws = torch.exp2(torch.arange(81).remainder(7).float() - 3).reshape(9, 9)
    pw = api.prepare_weight_b128(wq.to(torch.float8_e4m3fn).view(torch.uint8).to(dev()), ws.to(dev()))
    y = api.linear(x.to(dev()), pw)
    _, _, A = ref.quantize(f64(x))
    scale = ref.spread(ws.numpy(), N, K)[np.arange(N), perm.numpy()]
    assert np.array_equal(f64(y), A[:, perm.numpy()] * scale)


@pytest.mark.parametrize("M", [3, 70])
def test_non_finite_activations_stay_in_their_rows(M):
    x = randn((M, 400), 6)
    x[1, 3] = float("inf")
    x[2, 399] = float("nan")
    wq, ws = make_weight(200, 400, 7)
    pw = api.prepare_weight_b128(wq.to(dev()), ws.to(dev()))
    y = api.linear(x.to(dev()), pw)
    assert y[1].isnan().all() and y[2].isnan().all()
    keep = [m for m in range(M) if m not in (1, 2)]
    check_linear(x[keep], wq, ws, None, y[keep])


@pytest.mark.parametrize("M", [4, 100])
def test_strided_operands_and_untouched_surroundings(M):
    N, K = 200, 528
    wide = spiky(M, 3 * K, 8).to(dev())
    x = wide[:, K:2 * K]                              # row stride 3 K, 16-byte aligned
    wq, ws = make_weight(N, K, 3)
    pw = api.prepare_weight_b128(wq.to(dev()), ws.to(dev()))
    out = torch.full((M + 2, N + 8), 7.0, dtype=torch.bfloat16, device=dev())
    y = api.linear(x, pw, out=out[1:M + 1, :N])
    check_linear(x.cpu(), wq, ws, None, y)
    edge = out.clone()
    edge[1:M + 1, :N] = 7.0
    assert (edge == 7.0).all()
    # columns that are not 16-byte aligned, a transposed and an expanded view
    odd = wide[:, 3:3 + K]
    check_linear(odd.cpu(), wq, ws, None, api.linear(odd, pw))
    tr = spiky(K, M, 2).to(dev()).t()
    check_linear(tr.cpu(), wq, ws, None, api.linear(tr, pw))
    ex = wide[:1, :K].expand(M, K)
    check_linear(ex.cpu(), wq, ws, None, api.linear(ex, pw))
    # leading dimensions
    assert torch.equal(api.linear(x.reshape(2, M // 2, K), pw).reshape(M, N), api.linear(x, pw))


def test_empty_batch():
    wq, ws = make_weight(64, 256, 3)
    pw = api.prepare_weight_b128(wq.to(dev()), ws.to(dev()))
    assert api.linear(torch.empty(0, 256, dtype=torch.bfloat16, device=dev()), pw).shape == (0, 64)


def test_same_result_twice_and_on_another_stream():
    x = spiky(300, 4096, 11).to(dev())
    wq, ws = make_weight(512, 4096, 12)
    pw = api.prepare_weight_b128(wq.to(dev()), ws.to(dev()))
    y = api.linear(x, pw)
    assert torch.equal(y, api.linear(x, pw))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        z = api.linear(x, pw)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(y, z)


@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_graph_replays(M):
    wq, ws = make_weight(512, 2064, 1)
    pw = api.prepare_weight_b128(wq.to(dev()), ws.to(dev()))
    x = spiky(M, 2064, 0).to(dev())
    api.linear(x, pw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = api.linear(x, pw)
    for seed in range(4):
        x.copy_(spiky(M, 2064, seed))
        want = api.linear(x, pw)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("tile", [64, 128, 256, 512])
@pytest.mark.parametrize("M,N,K", [(17, 8, 512), (128, 256, 528), (129, 264, 640), (300, 520, 1152), (700, 1024, 2064),
                                   (257, 136, 8336), (70, 264, 16),
                                   (140, 1032, 256), (100, 130, 640)])
def test_every_tile_form(tile, M, N, K):
    """Each tile form on shapes of one and many tiles, partial ones and a
    single weight group among them; persistent workgroups with several tiles."""
    x = spiky(M, K, M + N + K)
    wq, ws = make_weight(N, K, N + K)
    bias = randn((N,), 9)
    pw = api.prepare_weight_b128(wq.to(dev()), ws.to(dev()))
    prev = api.mxfp8_debug_force_b128(tile)
    try:
        out = torch.full((M + 1, N + 16), 3.0, dtype=torch.bfloat16, device=dev())
        y = api.linear(x.to(dev()), pw, bias.to(dev()), out=out[:M, :N])
        z = api.linear(x.to(dev()), pw, bias.to(dev()))
    finally:
        api.mxfp8_debug_force_b128(prev)
    check_linear(x, wq, ws, bias, y)
    assert torch.equal(y, z)
    assert (out[M] == 3.0).all() and (out[:, N:] == 3.0).all()


def test_many_tiles_per_workgroup():
    """More large tiles than compute units: the pipeline runs from tile to
    tile.  Every output against the small tiles', and a sample of rows against
    64 bits."""
    M, N, K = 4200, 4360, 640
    x, (wq, ws) = spiky(M, K, 1), make_weight(N, K, 2)
    pw = api.prepare_weight_b128(wq.to(dev()), ws.to(dev()))
    bias = randn((N,), 3).to(dev())
    y = {}
    for tile in (128, 256, 512):
        prev = api.mxfp8_debug_force_b128(tile)
        try:
            y[tile] = api.linear(x.to(dev()), pw, bias)
        finally:
            api.mxfp8_debug_force_b128(prev)
    assert torch.equal(y[128], y[256]) and torch.equal(y[128], y[512])    # the same blocks in the same order
    rows = torch.arange(0, M, 97)
    check_linear(x[rows], wq, ws, bias.cpu(), y[256][rows.to(dev())])


@pytest.mark.parametrize("M,N,K", [(1, 28672, 1040), (9, 300, 2048), (16, 40, 2064), (17, 1, 16), (18, 130, 2048),
                                   (24, 515, 2064), (32, 4000, 4096), (31, 100, 8208), (32, 264, 16400), (25, 16400, 2048),
                                   (32, 70000, 1024), (16, 70000, 4096)])
def test_few_rows(M, N, K):
    """One and two groups of sixteen rows, turns of one, two and four blocks,
    and sizes whose few rows take the tiles."""
    x = spiky(M, K, M + K)
    wq, ws = make_weight(N, K, N)
    bias = randn((N,), 4)
    pw = api.prepare_weight_b128(wq.to(dev()), ws.to(dev()))
    y = api.linear(x.to(dev()), pw, bias.to(dev()))
    check_linear(x, wq, ws, bias, y)
    assert torch.equal(y, api.linear(x.to(dev()), pw, bias.to(dev())))
    # strides, and the surroundings of y
    wide = torch.full((M + 2, N + 13), 7.0, dtype=torch.bfloat16, device=dev())
    xs = torch.zeros(M, K + 24, dtype=torch.bfloat16, device=dev())
    xs[:, 8:8 + K] = x.to(dev())
    api.linear(xs[:, 8:8 + K], pw, bias.to(dev()), out=wide[1:1 + M, 5:5 + N])
    assert torch.equal(wide[1:1 + M, 5:5 + N], y)
    wide[1:1 + M, 5:5 + N] = 7.0
    assert bool((wide == 7.0).all())


@pytest.mark.parametrize("M", [20, 32])
def test_two_row_groups_place_every_element(M):
    """One-hot weights: y[m, n] is one dequantized activation."""
    K = N = 272
    x = spiky(M, K, 3)
    q = torch.eye(N).to(torch.float8_e4m3fn).view(torch.uint8)
    pw = api.prepare_weight_b128(q.to(dev()), torch.ones(3, 3, device=dev()))
    _, _, A = ref.quantize(f64(x))
    assert np.array_equal(f64(api.linear(x.to(dev()), pw)), A)


def test_non_finite_rows_of_two_groups():
    x = randn((30, 512), 1)
    x[3, 5], x[20, 300] = float("inf"), float("nan")
    wq, ws = make_weight(64, 512, 2)
    y = api.linear(x.to(dev()), api.prepare_weight_b128(wq.to(dev()), ws.to(dev()))).cpu()
    bad = torch.zeros(30, dtype=torch.bool)
    bad[[3, 20]] = True
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()
