"""Plain 64-bit forms of the MXFP4 layer, for its tests."""

import numpy as np
import torch

import oracle
from mxfp8_block_scaled_amd import api, synth


def activations(M, K, seed, std=1.0):
    return synth.randn_bf16((M, K), std, torch.Generator().manual_seed(seed))


def weight(N, K, seed, std=0.02):
    """(codes, scale bytes, dequantized values) of a random MXFP4 weight."""
    w = synth.randn_bf16((N, K), std, torch.Generator().manual_seed(seed)).double().numpy()
    codes, s = oracle.quantize_mxfp4(w)
    packed = oracle.pack_fp4(codes)
    return packed, s, oracle.dequantize_mxfp4(packed, s)


def quantized(x):
    """What bf16 rows are worth after 4-bit quantization; NaN in blocks with an
    infinity or a NaN."""
    x = x.double().numpy()
    blocks = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(blocks).all(axis=2)
    codes, s = oracle.quantize_mxfp4(np.where(bad[:, :, None], 0.0, blocks).reshape(x.shape))
    A = oracle.dequantize_mxfp4(oracle.pack_fp4(codes), s).reshape(blocks.shape)
    return np.where(bad[:, :, None], np.nan, A).reshape(x.shape)


def bound(A, W, r):
    """Bound of |y - r| for operands A [M, K] and W [N, K].  Each scaled MFMA (128
    elements) is off by at most 2^-10 of its largest product (measured for
    8-bit operands: 2^-12; 4-bit ones have shorter products); the fp32 sums
    round K times by at most 2^-23 of the sum of magnitudes; one rounding to
    bf16 is half a step, 2^-8 relative."""
    K = A.shape[1]
    amax, wmax = np.abs(A).max(axis=1, initial=0), np.abs(W).max(axis=1, initial=0)
    acc = K / 128.0 * 2.0 ** -10 * np.outer(amax, wmax) + K * 2.0 ** -23 * (np.abs(A) @ np.abs(W).T)
    return 2.0 ** -8 * np.abs(r) + (1 + 2.0 ** -8) * acc + 2.0 ** -133


def check(y, A, W, bias=None):
    """y (bf16 tensor) against the product of the quantized operands."""
    r = A @ W.T
    if bias is not None:
        r = r + bias.double().numpy()
    y = y.double().cpu().numpy()
    assert y.shape == r.shape
    over = ~(np.abs(y - r) <= bound(A, W, r))
    assert not over.any(), (int(over.sum()), np.argwhere(over)[:4].tolist(), y[over][:4], r[over][:4])


class forced:
    def __init__(self, form):
        self.form = form

    def __enter__(self):
        self.before = api.mxfp8_debug_force_w4a4(self.form)

    def __exit__(self, *_):
        api.mxfp8_debug_force_w4a4(self.before)
