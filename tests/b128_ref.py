"""Plain 64-bit forms of the 128-block quantization, used by its tests."""

import numpy as np
import torch


def scale_bytes(amax):
    """UE8M0 byte of the smallest power of two s with amax / s <= 448; 0 for a
    zero or tiny maximum, 0xFF where the maximum is not finite."""
    amax = np.asarray(amax, dtype=np.float64)
    finite = np.isfinite(amax)
    m, e = np.frexp(np.where(finite & (amax > 0), amax, 1.0))
    j = e - 9 + (m > 448.0 / 512.0)
    byte = np.maximum(j + 127, 0)
    byte = np.where(amax == 0, 0, byte)
    return np.where(finite, byte, 255).astype(np.uint8)


def e4m3_round(v):
    """Nearest E4M3 value, ties to even (|v| <= 448)."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(np.maximum(np.abs(v), 2.0 ** -6))
    step = np.exp2(e - 4.0)
    return np.rint(v / step) * step


def quantize(x, rows=1):
    """x float64 [R, K] -> (values on the E4M3 grid, scale bytes
    [ceil(R / rows), ceil(K / 128)], dequantized values)."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    rb, kb = -(-R // rows), -(-K // 128)
    pad = np.zeros((rb * rows, kb * 128))
    pad[:R, :K] = x
    t = pad.reshape(rb, rows, kb, 128)
    s = scale_bytes(np.abs(t).max(axis=(1, 3)))
    val = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))[:, None, :, None]
    q = e4m3_round(t / val)
    back = lambda a: np.broadcast_to(a, t.shape).reshape(rb * rows, kb * 128)[:R, :K]
    return back(q), s, back(q * val)


def decode(q_bytes):
    return torch.as_tensor(q_bytes).view(torch.float8_e4m3fn).double().numpy()


def spread(s, N, K):
    """Block scales [.., ..] -> [N, K]."""
    return np.repeat(np.repeat(np.asarray(s, dtype=np.float64), 128, 0)[:N], 128, 1)[:, :K]


def gemm_bound(A, W, terms=64.0):
    """Bound of the GEMM's error before the output rounding, for operands A
    [M, K] and W [N, K]: each scaled MFMA is off by at most 2^-10 of its
    largest product (measured: 2^-12) and there is one per 128 elements (the
    bound allows one per 64); its scaling and the fp32 additions round K times
    by at most 2^-23 of the sum of magnitudes."""
    K = A.shape[1]
    amax, wmax = np.abs(A).max(axis=1, initial=0), np.abs(W).max(axis=1, initial=0)
    acc = max(1.0, K / terms) * 2.0 ** -10 * np.outer(amax, wmax) + (K + 16) * 2.0 ** -23 * (np.abs(A) @ np.abs(W).T)
    return (1 + 2.0 ** -8) * acc + 2.0 ** -133
