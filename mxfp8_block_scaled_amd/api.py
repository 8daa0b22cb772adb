"""Thin Python binding over libmxfp8.so (ctypes).

Argument marshalling only: torch tensors supply device memory and the current
HIP stream; every step of the layer runs in the library's HIP kernels.  If the
library has not been built, the first call raises ``MXFP8Error``; there is no
fallback.

Names mirror the C ABI (include/mxfp8.h): ``mxfp8_quantize_act``,
``mxfp8_prepare_weight``, ``mxfp8_linear``, ... take raw pointers and sizes;
``quantize_act``, ``prepare_weight`` and ``linear`` are the tensor-level
wrappers (the apply path of vLLM PR #52204: assert bf16, view the input as
``[-1, K]``, run the layer, restore the leading dims).
"""

import contextlib
import ctypes
import functools
import os
import threading

import torch
from torch.autograd import forward_ad

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libmxfp8.so")
_lib = None
_lock = threading.Lock()

_i64 = ctypes.c_int64
_vp = ctypes.c_void_p
_sz = ctypes.c_size_t

_SIGNATURES = {
    "mxfp8_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "mxfp8_quantize_act": ([_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp], ctypes.c_int),
    "mxfp8_prepared_weight_bytes": ([_i64, _i64, ctypes.POINTER(_sz), ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_prepare_weight": ([_vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp], ctypes.c_int),
    "mxfp8_unpack_weight": ([_vp, _vp, _i64, _i64, _vp, _vp, _vp], ctypes.c_int),
    "mxfp8_linear_workspace_bytes": ([_i64, _i64, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_linear": ([_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _vp, _sz, _vp], ctypes.c_int),
    "mxfp8_packed_act_bytes": ([_i64, _i64, ctypes.POINTER(_sz), ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_quantize_act_packed": ([_vp, _i64, _i64, _i64, _vp, _vp, _vp], ctypes.c_int),
    "mxfp8_gemm_packed": ([_vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _vp], ctypes.c_int),
    "mxfp8_debug_force_path": ([ctypes.c_int], ctypes.c_int),
    "mxfp8_debug_plan": ([_i64, _i64, _i64, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)], ctypes.c_int),
    "mxfp8_moe_prepared_bytes": ([_i64, _i64, _i64, ctypes.POINTER(_sz), ctypes.POINTER(_sz),
                                  ctypes.POINTER(_sz), ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_moe_prepare_weights": ([_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
    "mxfp8_moe_workspace_bytes": ([_i64, _i64, _i64, _i64, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_moe_grouped": ([_vp, _vp, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
                          ctypes.c_int),
    "mxfp8_moe_debug_capture": ([_vp, _vp, _vp, _vp, _vp], ctypes.c_int),
    "mxfp8_quantize_fp4": ([_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp], ctypes.c_int),
    "mxfp8_prepared_weight_fp4_bytes": ([_i64, _i64, ctypes.POINTER(_sz), ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_prepare_weight_fp4": ([_vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp], ctypes.c_int),
    "mxfp8_unpack_weight_fp4": ([_vp, _vp, _i64, _i64, _vp, _vp, _vp], ctypes.c_int),
    "mxfp8_linear_w4a8_workspace_bytes": ([_i64, _i64, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_linear_w4a8": ([_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _vp, _sz, _vp], ctypes.c_int),
    "mxfp8_linear_noalloc": ([_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _vp], ctypes.c_int),
    "mxfp8_gemm_prequant_workspace_bytes": ([_i64, _i64, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_gemm_prequant": ([_vp, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _vp, _sz, _vp],
                            ctypes.c_int),
    "mxfp8_quantize_b128": ([_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp], ctypes.c_int),
    "mxfp8_packed_act_b128_bytes": ([_i64, _i64, ctypes.POINTER(_sz), ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_quantize_act_packed_b128": ([_vp, _i64, _i64, _i64, _vp, _vp, _vp], ctypes.c_int),
    "mxfp8_dequantize_act_packed": ([_vp, _vp, _i64, _i64, _vp, _i64, _vp], ctypes.c_int),
    "mxfp8_prepared_weight_b128_bytes": ([_i64, _i64, ctypes.POINTER(_sz), ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_prepare_weight_b128": ([_vp, _vp, _i64, _i64, _i64, _i64, ctypes.c_int, _vp, _vp, _vp], ctypes.c_int),
    "mxfp8_quantize_weight_b128": ([_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp],
                                   ctypes.c_int),
    "mxfp8_linear_b128_workspace_bytes": ([_i64, _i64, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_linear_b128": ([_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _vp, _sz, _vp], ctypes.c_int),
    "mxfp8_gemm_packed_b128_workspace_bytes": ([_i64, _i64, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_gemm_packed_b128": ([_vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _vp, _sz, _vp], ctypes.c_int),
    "mxfp8_linear_b128_layer_bytes": ([_i64, _i64, _i64, ctypes.c_int, ctypes.POINTER(_sz), ctypes.POINTER(_sz),
                                       ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_linear_b128_forward": ([_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, ctypes.c_int, _vp, _vp, _sz,
                                   _vp], ctypes.c_int),
    "mxfp8_linear_b128_backward": ([_vp, _i64, _i64, _i64, _i64, ctypes.c_int, _vp, _vp, _i64, _vp, ctypes.c_int, _i64,
                                    _vp, ctypes.c_int, _vp, _sz, _vp], ctypes.c_int),
    "mxfp8_debug_force_b128": ([ctypes.c_int], ctypes.c_int),
    "mxfp8_debug_force_wgrad": ([ctypes.c_int], ctypes.c_int),
    "mxfp8_linear_wgrad_workspace_bytes": ([_i64, _i64, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_linear_wgrad": ([_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, ctypes.c_int, _i64, _vp, ctypes.c_int,
                            ctypes.c_int, _vp, _sz, _vp], ctypes.c_int),
    "mxfp8_moe_balance_workspace_bytes": ([_i64, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_moe_balance": ([_vp, ctypes.c_int, _i64, _i64, _i64, _i64, _vp, ctypes.c_float, ctypes.c_float, _vp, _vp,
                           _vp, _vp, _sz, _vp], ctypes.c_int),
    "mxfp8_moe_balance_backward": ([_vp, ctypes.c_int, _i64, _i64, _i64, _i64, _vp, ctypes.c_float, ctypes.c_float,
                                    _vp, _vp, _vp, _vp, _i64, _vp], ctypes.c_int),
    "mxfp8_packed_act_fp4_bytes": ([_i64, _i64, ctypes.POINTER(_sz), ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_quantize_act_packed_fp4": ([_vp, _i64, _i64, _i64, _vp, _vp, _vp], ctypes.c_int),
    "mxfp8_gemm_packed_fp4": ([_vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _vp], ctypes.c_int),
    "mxfp8_linear_w4a4_workspace_bytes": ([_i64, _i64, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_linear_w4a4": ([_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _vp, _sz, _vp], ctypes.c_int),
    "mxfp8_debug_force_w4a4": ([ctypes.c_int], ctypes.c_int),
    "mxfp8_moe_sort_workspace_bytes": ([_i64, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_moe_sort": ([_vp, ctypes.c_int, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "mxfp8_moe_permute": ([_vp, ctypes.c_int, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp], ctypes.c_int),
    "mxfp8_moe_unpermute": ([_vp, ctypes.c_int, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _vp], ctypes.c_int),
    "mxfp8_moe_unpermute_backward": ([_vp, ctypes.c_int, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _i64,
                                      _vp, _vp], ctypes.c_int),
    "mxfp8_moe_prepared_experts_fp4_bytes": ([_i64, _i64, _i64, ctypes.POINTER(_sz), ctypes.POINTER(_sz)],
                                             ctypes.c_int),
    "mxfp8_moe_prepare_experts_fp4": ([_vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp], ctypes.c_int),
    "mxfp8_moe_linear_w4a4_workspace_bytes": ([_i64, _i64, _i64, _i64, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "mxfp8_moe_linear_w4a4": ([_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _sz,
                               _vp], ctypes.c_int),
}

# Static scratch of mxfp8_linear_noalloc (bytes; MXFP8_NOALLOC_SCRATCH_BYTES).
NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024


class MXFP8Error(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = lib().mxfp8_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{where}: {msg} (status {status})")


def lib_path():
    return _LIB_PATH


def lib():
    """Load libmxfp8.so once; raise if it is missing."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(_LIB_PATH):
                    raise RuntimeError(
                        f"libmxfp8.so not built at {_LIB_PATH}; run "
                        "`python -m mxfp8_block_scaled_amd.build` (hipcc, gfx950)")
                handle = ctypes.CDLL(_LIB_PATH)
                for name, (args, res) in _SIGNATURES.items():
                    fn = getattr(handle, name)
                    fn.argtypes = args
                    fn.restype = res
                _lib = handle
    return _lib


def _check(status, where):
    if status != 0:
        raise MXFP8Error(status, where)


def _stream(device=None):
    """Handle of the device's current stream (an int; the Stream object that
    torch.cuda.current_stream builds costs more than a small kernel)."""
    index = None if device is None else device.index
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if index is None else index)


def _ptr(t):
    return None if t is None else t.data_ptr()


# ---------------------------------------------------------------------------
# Raw C-ABI mirrors (pointers are ints or None; stream is an int handle)
# ---------------------------------------------------------------------------

def mxfp8_status_string(status):
    return lib().mxfp8_status_string(status).decode()


def mxfp8_quantize_act(x, M, K, ldx, q, ldq, s, lds, stream):
    return lib().mxfp8_quantize_act(x, M, K, ldx, q, ldq, s, lds, stream)


def mxfp8_prepared_weight_bytes(N, K):
    w, s = _sz(), _sz()
    _check(lib().mxfp8_prepared_weight_bytes(N, K, ctypes.byref(w), ctypes.byref(s)),
           "mxfp8_prepared_weight_bytes")
    return w.value, s.value


def mxfp8_prepare_weight(w, ws, N, K, ldw, ldws, wp, sp, stream):
    return lib().mxfp8_prepare_weight(w, ws, N, K, ldw, ldws, wp, sp, stream)


def mxfp8_unpack_weight(wp, sp, N, K, w, ws, stream):
    return lib().mxfp8_unpack_weight(wp, sp, N, K, w, ws, stream)


def mxfp8_linear_workspace_bytes(M, N, K):
    b = _sz()
    _check(lib().mxfp8_linear_workspace_bytes(M, N, K, ctypes.byref(b)), "mxfp8_linear_workspace_bytes")
    return b.value


def mxfp8_linear(x, M, K, ldx, wp, sp, N, bias, y, ldy, ws, ws_bytes, stream):
    return lib().mxfp8_linear(x, M, K, ldx, wp, sp, N, bias, y, ldy, ws, ws_bytes, stream)


def mxfp8_linear_noalloc(x, M, K, ldx, wp, sp, N, bias, y, ldy, stream):
    return lib().mxfp8_linear_noalloc(x, M, K, ldx, wp, sp, N, bias, y, ldy, stream)


def mxfp8_quantize_fp4(x, M, K, ldx, q, ldq, s, lds, stream):
    return lib().mxfp8_quantize_fp4(x, M, K, ldx, q, ldq, s, lds, stream)


def quantize_fp4(x):
    """bf16 ``[M, K]`` (GPU) -> (uint8 ``[M, K/2]`` packed E2M1, uint8 ``[M, K/32]``
    UE8M0), the MX rule with E2M1 elements."""
    assert x.dtype == torch.bfloat16
    _require_cuda(x, "x")
    if x.stride(-1) != 1 or x.stride(0) % 8 != 0 or x.data_ptr() % 16 != 0:
        x = x.contiguous()
    M, K = x.shape
    q = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
    s = torch.empty((M, K // 32), dtype=torch.uint8, device=x.device)
    _check(mxfp8_quantize_fp4(_ptr(x), M, K, x.stride(0), _ptr(q), q.stride(0), _ptr(s), s.stride(0),
                              _stream(x.device)), "mxfp8_quantize_fp4")
    return q, s


def mxfp8_prepared_weight_fp4_bytes(N, K):
    w, s = _sz(), _sz()
    _check(lib().mxfp8_prepared_weight_fp4_bytes(N, K, ctypes.byref(w), ctypes.byref(s)),
           "mxfp8_prepared_weight_fp4_bytes")
    return w.value, s.value


def mxfp8_prepare_weight_fp4(w, ws, N, K, ldw, ldws, wp, sp, stream):
    return lib().mxfp8_prepare_weight_fp4(w, ws, N, K, ldw, ldws, wp, sp, stream)


def mxfp8_unpack_weight_fp4(wp, sp, N, K, w, ws, stream):
    return lib().mxfp8_unpack_weight_fp4(wp, sp, N, K, w, ws, stream)


def mxfp8_linear_w4a8_workspace_bytes(M, N, K):
    b = _sz()
    _check(lib().mxfp8_linear_w4a8_workspace_bytes(M, N, K, ctypes.byref(b)), "mxfp8_linear_w4a8_workspace_bytes")
    return b.value


def mxfp8_linear_w4a8(x, M, K, ldx, wp, sp, N, bias, y, ldy, ws, ws_bytes, stream):
    return lib().mxfp8_linear_w4a8(x, M, K, ldx, wp, sp, N, bias, y, ldy, ws, ws_bytes, stream)


def mxfp8_packed_act_bytes(M, K):
    q, s = _sz(), _sz()
    _check(lib().mxfp8_packed_act_bytes(M, K, ctypes.byref(q), ctypes.byref(s)), "mxfp8_packed_act_bytes")
    return q.value, s.value


def mxfp8_quantize_act_packed(x, M, K, ldx, qp, sp, stream):
    return lib().mxfp8_quantize_act_packed(x, M, K, ldx, qp, sp, stream)


def mxfp8_gemm_packed(qp, sp, M, K, wp, wsp, N, bias, y, ldy, stream):
    return lib().mxfp8_gemm_packed(qp, sp, M, K, wp, wsp, N, bias, y, ldy, stream)


def mxfp8_gemm_prequant_workspace_bytes(M, N, K):
    b = _sz()
    _check(lib().mxfp8_gemm_prequant_workspace_bytes(M, N, K, ctypes.byref(b)), "mxfp8_gemm_prequant_workspace_bytes")
    return b.value


def mxfp8_gemm_prequant(q, ldq, s, lds, M, K, wp, wsp, N, bias, y, ldy, ws, ws_bytes, stream):
    return lib().mxfp8_gemm_prequant(q, ldq, s, lds, M, K, wp, wsp, N, bias, y, ldy, ws, ws_bytes, stream)


def gemm_prequant(q, s, pw, bias=None):
    """The block-scaled GEMM + epilogue on row-major quantized activations
    (uint8 E4M3 ``q[M, K]``, UE8M0 ``s[M, >= K/32]``, GPU): bf16 ``[M, N]``."""
    _one_weight(pw)
    if isinstance(pw, PreparedWeightB128):
        raise ValueError("gemm_prequant takes an MXFP8 weight, not one with 128-blocks")
    if isinstance(pw, PreparedWeightFP4):
        raise ValueError("gemm_prequant takes an MXFP8 weight, not an MXFP4 one")
    q = _as_bytes(q)
    s = _as_bytes(s)
    _require_cuda(q, "q")
    if q.stride(-1) != 1 or q.stride(0) % 16 != 0 or q.data_ptr() % 16 != 0:
        q = q.contiguous()
    if s.stride(-1) != 1:
        s = s.contiguous()
    M, K = q.shape
    assert K == pw.K
    y = torch.empty((M, pw.N), dtype=torch.bfloat16, device=q.device)
    ws = torch.empty(mxfp8_gemm_prequant_workspace_bytes(M, pw.N, K), dtype=torch.uint8, device=q.device)
    _check(mxfp8_gemm_prequant(_ptr(q), q.stride(0), _ptr(s), s.stride(0), M, K, _ptr(pw.w_packed), _ptr(pw.s_packed),
                               pw.N, _ptr(bias), _ptr(y), y.stride(0), _ptr(ws), ws.numel(), _stream(q.device)),
           "mxfp8_gemm_prequant")
    return y


def mxfp8_debug_force_path(path):
    return lib().mxfp8_debug_force_path(path)


def mxfp8_debug_plan(M, N, K):
    """(path, splits) mxfp8_linear takes for M x N x K: path 0 = large-tile
    GEMM, 1 = decode kernel, 2 = mid-M kernel."""
    p, sp = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().mxfp8_debug_plan(M, N, K, ctypes.byref(p), ctypes.byref(sp)), "mxfp8_debug_plan")
    return p.value, sp.value


# ---------------------------------------------------------------------------
# Tensor-level API
# ---------------------------------------------------------------------------

def _require_cuda(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")


def quantize_act(x):
    """bf16 ``x[M, K]`` (GPU) -> (E4M3 bytes uint8 ``[M, K]``, UE8M0 bytes uint8 ``[M, K/32]``)."""
    assert x.dtype == torch.bfloat16, f"MXFP8 quantization takes bfloat16, got {x.dtype}"
    _require_cuda(x, "x")
    x2 = x.reshape(-1, x.shape[-1])
    if x2.stride(-1) != 1:
        x2 = x2.contiguous()
    M, K = x2.shape
    q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    s = torch.empty((M, K // 32), dtype=torch.uint8, device=x.device)
    _check(mxfp8_quantize_act(_ptr(x2), M, K, x2.stride(0), _ptr(q), K, _ptr(s), K // 32,
                              _stream(x.device)), "mxfp8_quantize_act")
    return q, s


class PreparedWeight:
    """An MXFP8 weight after the one-time preparation: packed payload and
    scales (opaque layout, N padded to 128) plus the logical output size."""

    def __init__(self, w_packed, s_packed, N, K):
        self.w_packed = w_packed
        self.s_packed = s_packed
        self.N = N
        self.K = K

    @property
    def device(self):
        return self.w_packed.device

    def unpack(self):
        """(E4M3 ``[N_pad, K]``, UE8M0 ``[N_pad, K/32]``) as uint8 tensors."""
        n_pad = (self.N + 127) // 128 * 128
        w = torch.empty((n_pad, self.K), dtype=torch.uint8, device=self.device)
        s = torch.empty((n_pad, self.K // 32), dtype=torch.uint8, device=self.device)
        _check(mxfp8_unpack_weight(_ptr(self.w_packed), _ptr(self.s_packed), self.N, self.K, _ptr(w), _ptr(s),
                                   _stream(self.device)), "mxfp8_unpack_weight")
        return w, s


def _one_weight(pw):
    """Refuses experts' weights, which have a single weight's fields."""
    if isinstance(pw, ExpertWeightsFP4):
        raise ValueError("experts' weights go to moe_linear_w4a4: this takes one MXFP8 weight, or one of another format")


def _as_bytes(t):
    return t.view(torch.uint8) if t.dtype != torch.uint8 else t


def prepare_weight(w_q, w_s):
    """MXFP8 weight ``w_q`` E4M3 ``[N, K]`` (uint8 or float8_e4m3fn) with UE8M0
    scales ``w_s`` ``[>= N, >= K/32]`` (uint8) -> PreparedWeight."""
    w_q = _as_bytes(w_q)
    w_s = _as_bytes(w_s)
    _require_cuda(w_q, "w_q")
    N, K = w_q.shape
    if w_q.stride(-1) != 1:
        w_q = w_q.contiguous()
    if w_s.stride(-1) != 1:
        w_s = w_s.contiguous()
    wb, sb = mxfp8_prepared_weight_bytes(N, K)
    wp = torch.empty(wb, dtype=torch.uint8, device=w_q.device)
    sp = torch.empty(sb, dtype=torch.uint8, device=w_q.device)
    _check(mxfp8_prepare_weight(_ptr(w_q), _ptr(w_s), N, K, w_q.stride(0), w_s.stride(0), _ptr(wp), _ptr(sp),
                                _stream(w_q.device)), "mxfp8_prepare_weight")
    return PreparedWeight(wp, sp, N, K)


_workspaces = {}
# Buffers a larger shape replaced.  They are never freed: a HIP graph captured
# earlier, or work still queued on the stream, may hold their addresses.
_retired = []


def _cache_key(device, stream):
    d = torch.device(device)
    idx = d.index if d.index is not None else torch.cuda.current_device()
    return idx, int(stream.cuda_stream)


def workspace(M, N, K, device):
    """A zero-initialised workspace big enough for mxfp8_linear at (M, N, K),
    cached per (device, current stream) and grown on demand (allocation
    happens here, never in the library).  Calls sharing a workspace must be
    ordered on one stream, hence one buffer per stream; a buffer that a
    larger shape replaces stays allocated for the life of the process, so a
    captured graph or queued work that still uses it never sees freed memory."""
    return _workspace_sized(mxfp8_linear_workspace_bytes(M, N, K), device)


def _workspace_sized(need, device, cache=None, zero=True):
    cache = _workspaces if cache is None else cache
    key = _cache_key(device, torch.cuda.current_stream(device))
    ws = cache.get(key)
    if ws is None or ws.numel() < need:
        if ws is not None:
            _retired.append(ws)
        size = max(need, 256)
        ws = torch.zeros(size, dtype=torch.uint8, device=device) if zero else \
            torch.empty(size, dtype=torch.uint8, device=device)
        cache[key] = ws
    return ws


class PreparedWeightFP4(PreparedWeight):
    """An MXFP4 weight after the one-time preparation (packed E2M1 payload,
    N_pad * K / 2 bytes, and its UE8M0 scales)."""

    def unpack(self):
        """(E2M1 ``[N_pad, K/2]``, two codes per byte, UE8M0 ``[N_pad, K/32]``)
        as uint8 tensors."""
        n_pad = (self.N + 127) // 128 * 128
        w = torch.empty((n_pad, self.K // 2), dtype=torch.uint8, device=self.device)
        s = torch.empty((n_pad, self.K // 32), dtype=torch.uint8, device=self.device)
        _check(mxfp8_unpack_weight_fp4(_ptr(self.w_packed), _ptr(self.s_packed), self.N, self.K, _ptr(w), _ptr(s),
                                       _stream(self.device)), "mxfp8_unpack_weight_fp4")
        return w, s


def prepare_weight_fp4(w_e2m1, w_s):
    """MXFP4 weight: ``w_e2m1`` uint8 ``[N, K/2]`` (two E2M1 codes per byte,
    element 2j in the low nibble) with UE8M0 scales ``w_s`` ``[>= N, >= K/32]``
    -> PreparedWeightFP4."""
    w_e2m1 = _as_bytes(w_e2m1)
    w_s = _as_bytes(w_s)
    _require_cuda(w_e2m1, "w_e2m1")
    N, K2 = w_e2m1.shape
    K = 2 * K2
    if w_e2m1.stride(-1) != 1 or w_e2m1.stride(0) % 16 != 0:
        w_e2m1 = w_e2m1.contiguous()
    if w_s.stride(-1) != 1:
        w_s = w_s.contiguous()
    wb, sb = mxfp8_prepared_weight_fp4_bytes(N, K)
    wp = torch.empty(wb, dtype=torch.uint8, device=w_e2m1.device)
    sp = torch.empty(sb, dtype=torch.uint8, device=w_e2m1.device)
    _check(mxfp8_prepare_weight_fp4(_ptr(w_e2m1), _ptr(w_s), N, K, w_e2m1.stride(0), w_s.stride(0), _ptr(wp),
                                    _ptr(sp), _stream(w_e2m1.device)), "mxfp8_prepare_weight_fp4")
    return PreparedWeightFP4(wp, sp, N, K)


def linear(x, pw, bias=None, out=None, workspace=None):
    """The MXFP8 dense linear layer: ``y = bf16(deq(q(x)) @ deq(W).T + bias)``.

    ``x`` bf16 ``[..., K]`` (GPU), ``pw`` a PreparedWeight (MXFP8), a
    PreparedWeightFP4 (MXFP4, the W4A8 layer) or a PreparedWeightB128 (FP8
    with 128-blocks), ``bias`` bf16 ``[N]`` or None.  Returns bf16 ``[..., N]`` (contiguous).  ``workspace``: an
    optional uint8 GPU tensor of at least ``mxfp8_linear_workspace_bytes``
    (``mxfp8_linear_w4a8_workspace_bytes`` for MXFP4,
    ``mxfp8_linear_b128_workspace_bytes`` for 128-blocks) bytes, 256-byte
    aligned, owned by the caller; by default a cached buffer per (device,
    stream) is used (128-blocks: a fresh one from torch's allocator)."""
    _one_weight(pw)
    if isinstance(pw, PreparedWeightB128):
        return _linear_prepared_b128(x, pw, bias, out, workspace)
    assert x.dtype == torch.bfloat16, f"MXFP8 linear requires bfloat16 activations, got {x.dtype}"
    _require_cuda(x, "x")
    K = pw.K
    lead = x.shape[:-1]
    x2 = x.reshape(-1, K)
    if x2.stride(-1) != 1 or x2.stride(0) % 8 != 0 or x2.data_ptr() % 16 != 0:
        x2 = x2.contiguous()
    M = x2.shape[0]
    N = pw.N
    if bias is not None:
        assert bias.dtype == torch.bfloat16 and bias.numel() == N
        bias = bias.contiguous()
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if isinstance(pw, PreparedWeightFP4):
        ws = workspace if workspace is not None else \
            _workspace_sized(mxfp8_linear_w4a8_workspace_bytes(M, N, K), x.device)
        _check(mxfp8_linear_w4a8(_ptr(x2), M, K, x2.stride(0), _ptr(pw.w_packed), _ptr(pw.s_packed), N,
                                 _ptr(bias), _ptr(y), y.stride(0), _ptr(ws), ws.numel(), _stream(x.device)),
               "mxfp8_linear_w4a8")
        return y.view(*lead, N)
    ws = workspace if workspace is not None else _workspace_sized(mxfp8_linear_workspace_bytes(M, N, K), x.device)
    _check(mxfp8_linear(_ptr(x2), M, K, x2.stride(0), _ptr(pw.w_packed), _ptr(pw.s_packed), N, _ptr(bias),
                        _ptr(y), y.stride(0), _ptr(ws), ws.numel(), _stream(x.device)), "mxfp8_linear")
    return y.view(*lead, N)


class PackedActivation:
    """Activations quantized into the GEMM's packed operand layout (rows padded
    to 128): the first kernel of the large-M path."""

    def __init__(self, q_packed, s_packed, M, K, block=32):
        self.q_packed = q_packed
        self.s_packed = s_packed
        self.M = M
        self.K = K
        self.block = block     # elements that share a scale: 32 (MX) or 128

    @property
    def device(self):
        return self.q_packed.device

    def dequantize(self):
        """The activations the 8-bit values stand for, bf16 ``[M, K]``."""
        x = torch.empty((self.M, self.K), dtype=torch.bfloat16, device=self.device)
        with _on(self.device):
            _check(lib().mxfp8_dequantize_act_packed(_ptr(self.q_packed), _ptr(self.s_packed), self.M, self.K,
                                                     _ptr(x), self.K, _stream(self.device)),
                   "mxfp8_dequantize_act_packed")
        return x

    def unpack(self):
        """(E4M3 ``[M_pad, K]``, UE8M0 ``[M_pad, K/32]``) as uint8 tensors
        (K % 256 == 0)."""
        return PreparedWeight(self.q_packed, self.s_packed, self.M, self.K).unpack()


def quantize_act_packed(x):
    """bf16 ``x[M, K]`` (GPU, K % 256 == 0) -> PackedActivation."""
    assert x.dtype == torch.bfloat16
    _require_cuda(x, "x")
    x2 = x.reshape(-1, x.shape[-1])
    if x2.stride(-1) != 1 or x2.stride(0) % 8 != 0 or x2.data_ptr() % 16 != 0:
        x2 = x2.contiguous()
    M, K = x2.shape
    qb, sb = mxfp8_packed_act_bytes(M, K)
    qp = torch.empty(qb, dtype=torch.uint8, device=x.device)
    sp = torch.empty(sb, dtype=torch.uint8, device=x.device)
    _check(mxfp8_quantize_act_packed(_ptr(x2), M, K, x2.stride(0), _ptr(qp), _ptr(sp), _stream(x.device)),
           "mxfp8_quantize_act_packed")
    return PackedActivation(qp, sp, M, K)


def gemm_packed(pa, pw, bias=None):
    """The GEMM + epilogue on packed activations (the second kernel of the
    large-M path), for activations and a weight of the same scale block."""
    _one_weight(pw)
    assert pa.K == pw.K
    b128 = isinstance(pw, PreparedWeightB128)
    fp4 = isinstance(pa, PackedActivationFP4)
    if pa.block != (128 if b128 else 32):
        raise ValueError(f"activations with a scale per {pa.block} elements do not go with this weight")
    if fp4 != isinstance(pw, PreparedWeightFP4):
        raise ValueError("MXFP4 activations and an MXFP4 weight go together")
    y = torch.empty((pa.M, pw.N), dtype=torch.bfloat16, device=pa.q_packed.device)
    if fp4:
        bias = _bias(bias, pw.N, align=4)
        _same_device(pa.q_packed, pw.w_packed, bias)
        with _on(pa.device):
            _check(lib().mxfp8_gemm_packed_fp4(_ptr(pa.q_packed), _ptr(pa.s_packed), pa.M, pa.K, _ptr(pw.w_packed),
                                               _ptr(pw.s_packed), pw.N, _ptr(bias), _ptr(y), y.stride(0),
                                               _stream(pa.device)), "mxfp8_gemm_packed_fp4")
        return y
    if b128:
        bias = _bias(bias, pw.N)
        _same_device(pa.q_packed, pw.w_packed, bias)
        with _on(pa.device):
            ws = _scratch(_bytes("mxfp8_gemm_packed_b128_workspace_bytes", pa.M, pw.N, pa.K), y)
            _check(lib().mxfp8_gemm_packed_b128(_ptr(pa.q_packed), _ptr(pa.s_packed), pa.M, pa.K, _ptr(pw.w_packed),
                                                _ptr(pw.s_packed), pw.N, _ptr(bias), _ptr(y), y.stride(0), _ptr(ws),
                                                ws.numel(), _stream(pa.device)), "mxfp8_gemm_packed_b128")
        return y
    _check(mxfp8_gemm_packed(_ptr(pa.q_packed), _ptr(pa.s_packed), pa.M, pa.K, _ptr(pw.w_packed),
                             _ptr(pw.s_packed), pw.N, _ptr(bias), _ptr(y), y.stride(0),
                             _stream(pa.q_packed.device)), "mxfp8_gemm_packed")
    return y


# ---------------------------------------------------------------------------
# FP8 with 128-blocks, and the layer's training side
# ---------------------------------------------------------------------------

_HERE_ALREADY = contextlib.nullcontext()


def _on(device):
    """Context in which ``device`` is the current one (the library launches on
    the current device)."""
    if device.index is None or device.index == torch.cuda.current_device():
        return _HERE_ALREADY
    return torch.cuda.device(device)


def _same_device(first, *rest):
    index = first.get_device()
    for t in rest:
        if t is not None and t.get_device() != index:
            raise ValueError(f"operands on {first.device} and {t.device}")


def _scratch(need, like):
    """A workspace on ``like``'s device for one call.  From torch's caching allocator each time, so
    that it follows the allocator's rules for streams and captured graphs: a
    graph keeps its own, and no two calls share one unless their order allows.
    None where none is needed."""
    return like.new_empty(need, dtype=torch.uint8) if need else None


@functools.lru_cache(maxsize=4096)
def _bytes(query, *sizes):
    """A host-only size query (a function of the sizes and the forced paths;
    the hooks that force one clear the cache)."""
    b = _sz()
    _check(getattr(lib(), query)(*sizes, ctypes.byref(b)), query)
    return b.value


def _rows(x, name):
    """bf16 ``[..., K]`` -> ``[M, K]`` as the library takes it: rows
    contiguous, 16-byte aligned, strides of whole 16 bytes."""
    if x.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16, got {x.dtype}")
    _require_cuda(x, name)
    x2 = x if x.dim() == 2 else x.reshape(-1, x.shape[-1])
    row, col = x2.stride()
    if col != 1 or row % 8 != 0 or row < x2.shape[1] or x2.data_ptr() % 16 != 0:
        x2 = x2.clone(memory_format=torch.contiguous_format)
    return x2


def _bias(bias, N, align=2):
    if bias is None:
        return None
    if bias.dtype != torch.bfloat16 or bias.numel() != N:
        raise ValueError(f"bias must be bfloat16 [{N}]")
    return bias.contiguous() if bias.data_ptr() % align == 0 else bias.clone(memory_format=torch.contiguous_format)


def mxfp8_linear_b128_workspace_bytes(M, N, K):
    return _bytes("mxfp8_linear_b128_workspace_bytes", M, N, K)


def mxfp8_linear_b128(x, M, K, ldx, wp, sp, N, bias, y, ldy, ws, ws_bytes, stream):
    return lib().mxfp8_linear_b128(x, M, K, ldx, wp, sp, N, bias, y, ldy, ws, ws_bytes, stream)


def mxfp8_debug_force_b128(tile):
    _bytes.cache_clear()
    _layer_bytes.cache_clear()
    return lib().mxfp8_debug_force_b128(tile)


def mxfp8_debug_force_wgrad(tile):
    _bytes.cache_clear()
    _layer_bytes.cache_clear()
    return lib().mxfp8_debug_force_wgrad(tile)


def mxfp8_prepared_weight_b128_bytes(N, K):
    w, s = _sz(), _sz()
    _check(lib().mxfp8_prepared_weight_b128_bytes(N, K, ctypes.byref(w), ctypes.byref(s)),
           "mxfp8_prepared_weight_b128_bytes")
    return w.value, s.value


class PreparedWeightB128(PreparedWeight):
    """An FP8 weight with an fp32 scale for each 128 x 128 block after the
    one-time preparation (packed E4M3 payload, rows and K padded to 128, and
    fp32 scales ``[ceil(N/128), ceil(K/128)]``)."""

    def unpack(self):
        raise NotImplementedError("128-block weights have no unpack entry")


def _empty_b128(N, K, device):
    wb, sb = mxfp8_prepared_weight_b128_bytes(N, K)
    return PreparedWeightB128(torch.empty(wb, dtype=torch.uint8, device=device),
                              torch.empty(sb // 4, dtype=torch.float32, device=device), N, K)


def prepare_weight_b128(w_q, w_s, transpose=False):
    """FP8 weight ``w_q`` E4M3 ``[N, K]`` (uint8 or float8_e4m3fn) with fp32
    scales ``w_s`` ``[ceil(N/128), ceil(K/128)]`` -> PreparedWeightB128.
    ``transpose``: of the transposed weight, for the input gradient
    ``linear(dy, prepared)``."""
    w_q = _as_bytes(w_q)
    _require_cuda(w_q, "w_q")
    _same_device(w_q, w_s)
    N, K = w_q.shape
    if w_s.dtype != torch.float32 or w_s.dim() != 2 or w_s.shape[0] < -(-N // 128) or w_s.shape[1] < -(-K // 128):
        raise ValueError(f"w_s must be float32 [{-(-N // 128)}, {-(-K // 128)}]")
    if w_q.stride(-1) != 1 or w_q.stride(0) % 16 != 0 or w_q.stride(0) < K or w_q.data_ptr() % 16 != 0:
        w_q = w_q.clone(memory_format=torch.contiguous_format)
    if w_s.stride(-1) != 1 or w_s.stride(0) < w_s.shape[1]:
        w_s = w_s.clone(memory_format=torch.contiguous_format)
    with _on(w_q.device):
        pw = _empty_b128(K, N, w_q.device) if transpose else _empty_b128(N, K, w_q.device)
        _check(lib().mxfp8_prepare_weight_b128(_ptr(w_q), _ptr(w_s), N, K, w_q.stride(0), w_s.stride(0),
                                               int(transpose), _ptr(pw.w_packed), _ptr(pw.s_packed),
                                               _stream(w_q.device)), "mxfp8_prepare_weight_b128")
    return pw


def _linear_prepared_b128(x, pw, bias, out, workspace):
    """``linear`` with a PreparedWeightB128."""
    x2 = _rows(x, "x")
    (M, K), N = x2.shape, pw.N
    if K != pw.K:
        raise ValueError(f"x has {K} columns, the weight {pw.K}")
    bias = _bias(bias, N)
    if out is None:
        out = x.new_empty(M, N)
    elif out.dtype != torch.bfloat16 or tuple(out.shape) != (M, N) or out.stride(1) != 1 or out.stride(0) < N:
        raise ValueError(f"out must be bfloat16 [{M}, {N}] with contiguous rows that do not overlap")
    _same_device(x2, pw.w_packed, bias, out, workspace)
    with _on(x.device):
        need = _bytes("mxfp8_linear_b128_workspace_bytes", M, N, K)
        ws = workspace if workspace is not None else _scratch(need, x)
        _check(lib().mxfp8_linear_b128(_ptr(x2), M, K, x2.stride(0), _ptr(pw.w_packed), _ptr(pw.s_packed), N,
                                       _ptr(bias), _ptr(out), out.stride(0), _ptr(ws), 0 if ws is None else ws.numel(),
                                       _stream(x.device)), "mxfp8_linear_b128")
    return out if x.dim() == 2 else out.view(*x.shape[:-1], N)


def quantize_weight_b128(w):
    """bf16 ``w[N, K]`` (GPU) -> (E4M3 bytes uint8 ``[N, K]``, fp32 scales
    ``[ceil(N/128), ceil(K/128)]``, powers of two)."""
    w = _rows(w, "w")
    N, K = w.shape
    q = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    s = torch.empty((-(-N // 128), -(-K // 128)), dtype=torch.float32, device=w.device)
    with _on(w.device):
        _check(lib().mxfp8_quantize_weight_b128(_ptr(w), N, K, w.stride(0), _ptr(q), K, _ptr(s), s.shape[1], None,
                                                None, None, None, _stream(w.device)), "mxfp8_quantize_weight_b128")
    return q, s


def prepare_weight_b128_bf16(w, transposed=True):
    """bf16 ``w[N, K]`` -> (PreparedWeightB128 of w, PreparedWeightB128 of
    w^T or None): ``quantize_weight_b128`` and ``prepare_weight_b128`` of both
    orientations in one pass over the weight."""
    w = _rows(w, "w")
    N, K = w.shape
    with _on(w.device):
        pw = _empty_b128(N, K, w.device)
        pt = _empty_b128(K, N, w.device) if transposed else None
        _check(lib().mxfp8_quantize_weight_b128(_ptr(w), N, K, w.stride(0), None, 0, None, 0, _ptr(pw.w_packed),
                                                _ptr(pw.s_packed), _ptr(pt.w_packed) if pt else None,
                                                _ptr(pt.s_packed) if pt else None, _stream(w.device)),
               "mxfp8_quantize_weight_b128")
    return pw, pt


def quantize_act_b128(x):
    """bf16 ``x[..., K]`` (GPU, K % 16 == 0) -> (E4M3 bytes uint8 ``[M, K]``,
    UE8M0 bytes uint8 ``[M, ceil(K/128)]``)."""
    x2 = _rows(x, "x")
    M, K = x2.shape
    q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    s = torch.empty((M, -(-K // 128)), dtype=torch.uint8, device=x.device)
    with _on(x.device):
        _check(lib().mxfp8_quantize_b128(_ptr(x2), M, K, x2.stride(0), _ptr(q), K, _ptr(s), s.shape[1],
                                         _stream(x.device)), "mxfp8_quantize_b128")
    return q, s


def quantize_act_packed_b128(x):
    """bf16 ``x[..., K]`` (GPU, K % 16 == 0) -> PackedActivation with a scale
    per 128 elements: the operand of ``gemm_packed`` and, kept until the
    backward pass, the 8-bit activation checkpoint ``linear_wgrad`` reads."""
    x2 = _rows(x, "x")
    M, K = x2.shape
    q, s = _sz(), _sz()
    _check(lib().mxfp8_packed_act_b128_bytes(max(M, 1), K, ctypes.byref(q), ctypes.byref(s)),
           "mxfp8_packed_act_b128_bytes")
    with _on(x.device):
        qp = torch.empty(q.value if M else 0, dtype=torch.uint8, device=x.device)
        sp = torch.empty(s.value if M else 0, dtype=torch.uint8, device=x.device)
        _check(lib().mxfp8_quantize_act_packed_b128(_ptr(x2), M, K, x2.stride(0), _ptr(qp), _ptr(sp),
                                                    _stream(x.device)), "mxfp8_quantize_act_packed_b128")
    return PackedActivation(qp, sp, M, K, block=128)


_DTYPES = {torch.float32: 0, torch.bfloat16: 1}   # mxfp8_dtype


def linear_wgrad(dy, pa, dtype=torch.float32, bias_grad=False, out=None, out_bias=None, accumulate=False):
    """Weight gradient from the 8-bit activation checkpoint ``pa`` (a
    PackedActivation of either 8-bit quantizer): ``dw[N, K] = dy^T deq(pa)``.

    ``dy`` bf16 ``[..., N]`` with M rows, N % 8 == 0.  Returns ``dw`` (``dtype``
    float32 or bfloat16; ``out`` if given), or ``(dw, db)`` with ``bias_grad``,
    ``db`` the column sums of dy (``out_bias``, float32 or bfloat16, if given,
    else fp32).  ``accumulate`` adds to ``out`` and ``out_bias`` (both fp32)
    instead of overwriting them."""
    if isinstance(pa, PackedActivationFP4):
        raise ValueError("the weight gradient takes 8-bit activations, not MXFP4 ones")
    d2 = _rows(dy, "dy")
    M, N = d2.shape
    if M != pa.M:
        raise ValueError(f"dy has {M} rows, the checkpoint {pa.M}")
    if accumulate and (out is None or (bias_grad and out_bias is None)):
        raise ValueError("accumulate needs the tensors to add to")
    if out is None:
        out = d2.new_empty((N, pa.K), dtype=dtype)
    if tuple(out.shape) != (N, pa.K) or out.dtype not in _DTYPES or out.stride(-1) != 1:
        raise ValueError(f"out must be float32 or bfloat16 [{N}, {pa.K}] with contiguous rows")
    db = None
    if bias_grad:
        db = out_bias if out_bias is not None else d2.new_empty(N, dtype=torch.float32)
        if db.dtype not in _DTYPES or tuple(db.shape) != (N,) or not db.is_contiguous():
            raise ValueError(f"out_bias must be contiguous float32 or bfloat16 [{N}]")
    if accumulate and (out.dtype != torch.float32 or (db is not None and db.dtype != torch.float32)):
        raise ValueError("accumulate needs float32 outputs")
    _same_device(d2, pa.q_packed, out, db)
    with _on(dy.device):
        need = _bytes("mxfp8_linear_wgrad_workspace_bytes", M, N, pa.K)
        ws = _scratch(need, d2)
        _check(lib().mxfp8_linear_wgrad(_ptr(d2), M, N, d2.stride(0), _ptr(pa.q_packed), _ptr(pa.s_packed), pa.K,
                                        _ptr(out), _DTYPES[out.dtype], out.stride(0), _ptr(db),
                                        0 if db is None else _DTYPES[db.dtype], int(accumulate), _ptr(ws), need,
                                        _stream(dy.device)), "mxfp8_linear_wgrad")
    return (out, db) if bias_grad else out


@functools.lru_cache(maxsize=4096)
def _layer_bytes(M, N, K, keep):
    """(kept, forward workspace, backward workspace) bytes of a training step."""
    out = [_sz() for _ in range(3)]
    _check(lib().mxfp8_linear_b128_layer_bytes(M, N, K, keep, *[ctypes.byref(o) for o in out]),
           "mxfp8_linear_b128_layer_bytes")
    return tuple(o.value for o in out)


def _linear_b128_forward(x, w, bias, keep):
    """(y, what the backward call needs, its workspace bytes) of a step that
    keeps what MXFP8_KEEP_DX (1) and MXFP8_KEEP_DW (2) in ``keep`` ask for."""
    x2, w2, bias = _rows(x, "x"), _rows(w, "w"), _bias(bias, w.shape[0])
    (M, K), N, d = x2.shape, w2.shape[0], x.device
    # in its last shape: of a view made in here, autograd refuses in-place use
    y = x.new_empty(M, N) if x.dim() == 2 else x.new_empty(*x.shape[:-1], N)
    with _on(d):
        kept_bytes, ws_bytes, back_bytes = _layer_bytes(M, N, K, keep)
        kept, ws = _scratch(kept_bytes, y), _scratch(ws_bytes, y)
        _check(lib().mxfp8_linear_b128_forward(_ptr(x2), M, K, x2.stride(0), _ptr(w2), N, w2.stride(0), _ptr(bias),
                                               _ptr(y), N, keep, _ptr(kept), _ptr(ws), ws_bytes, _stream(d)),
               "mxfp8_linear_b128_forward")
    return y, kept, back_bytes


# Captured backward passes.  A leaf's gradient accumulator belongs to the stream
# on which it was made and lives as long as some graph of that leaf, or something
# else that holds it.  A captured backward pass that hands it a gradient makes its
# stream wait for a captured event.  Any stream joins the capture by that but the
# legacy default one, which cannot, and the process ends.  So the accumulators'
# metadata note their streams, and a captured backward pass with one of the
# default stream, or of a stream that is not known, is refused.
_LEGACY, _UNKNOWN = 0, -1


def _mark_leaves_before(leaves, stream):
    """Before a node of these operands is made: accumulators that some other
    operator made are of an unknown stream.  (The mark goes with an accumulator
    that nothing holds.)  Not on the default stream, where the note would be
    the refused kind anyway: some microseconds per operand."""
    if stream == _LEGACY:
        return
    for t in leaves:
        if t is not None and t.requires_grad and t.is_leaf:
            torch.autograd.graph.get_gradient_edge(t).node.metadata.setdefault("mxfp8_stream", _UNKNOWN)


def _mark_leaves(out, stream):
    """Notes the stream of accumulators made with this node.  One of unknown
    stream shows it the first time that it runs, which torch does on its own
    stream."""
    for node, _ in out.grad_fn.next_functions:
        if not hasattr(node, "variable"):
            continue
        meta = node.metadata
        if meta.setdefault("mxfp8_stream", stream) == _UNKNOWN and "mxfp8_shows" not in meta:
            meta["mxfp8_shows"] = True
            device = node.variable.device
            node.register_prehook(lambda grads, meta=meta, device=device: meta.update(mxfp8_stream=_stream(device)))


def _check_capture(node, stream, capturing):
    """Raises where a captured backward pass of ``node`` would reach an
    accumulator of the default stream, or may."""
    if not capturing:
        return
    for n, _ in node.next_functions:
        if not hasattr(n, "variable"):
            continue
        of = n.metadata.get("mxfp8_stream", stream)
        if of != stream and of in (_LEGACY, _UNKNOWN):
            raise RuntimeError("backward pass captured while an earlier autograd graph of the same leaf tensors is "
                               "alive on another stream, the default one, or was made by another operator on a stream "
                               "that is not known: delete its outputs before the capture, and in the capture give "
                               "those leaves to this operator first")


def _reverse_only(name, *operands):
    """Refuses operands with a tangent in a call that goes past its node, since no
    reverse gradient is asked of it, and would lose them.  (The nodes refuse
    them by themselves.)"""
    # (outside of a level no tensor has one; where torch does not say, each is asked)
    if getattr(forward_ad, "_current_level", 0) < 0:
        return
    for t in operands:
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise RuntimeError(f"{name} is differentiable in reverse mode only")


class _LinearB128(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias):
        need_x, need_w, need_b = ctx.needs_input_grad
        ctx.keep = (1 if need_x else 0) | (2 if need_w or need_b else 0)
        y, kept, ctx.ws_bytes = _linear_b128_forward(x, w, bias, ctx.keep)
        ctx.save_for_backward(kept)   # freed with the graph's other saved tensors
        ctx.shape = x.shape
        return y

    @staticmethod
    def backward(ctx, dy):
        # (torch's wrapper, which makes second derivatives an error, costs a
        # small layer some microseconds and changes nothing in an ordinary pass)
        run = _LinearB128._differentiable_once if torch.is_grad_enabled() else _LinearB128._backward
        return run(ctx, dy)

    @staticmethod
    def _backward(ctx, dy):
        need_x, need_w, need_b = ctx.needs_input_grad
        kept, = ctx.saved_tensors
        d = dy.device
        stream = _stream(d)
        _check_capture(ctx, stream, torch.cuda.is_current_stream_capturing())
        d2 = _rows(dy, "dy")
        (M, N), K = d2.shape, ctx.shape[-1]
        dx = d2.new_empty(M, K) if need_x else None
        dw = d2.new_empty(N, K) if need_w or need_b else None
        db = d2.new_empty(N) if need_b else None
        with _on(d):
            ws = _scratch(ctx.ws_bytes, d2)
            _check(lib().mxfp8_linear_b128_backward(_ptr(d2), M, N, d2.stride(0), K, ctx.keep, _ptr(kept), _ptr(dx), K,
                                                    _ptr(dw), 1, K, _ptr(db), 1, _ptr(ws), ctx.ws_bytes, stream),
                   "mxfp8_linear_b128_backward")
        if need_x and len(ctx.shape) != 2:
            dx = dx.view(ctx.shape)
        return dx, dw if need_w else None, db

    _differentiable_once = staticmethod(torch.autograd.function.once_differentiable(_backward.__func__))


def linear_b128(x, w, bias=None):
    """The 128-block FP8 linear layer from a bf16 weight, with gradients:
    ``y = bf16(deq(q(x)) @ deq(q(w)).T + bias)``, x ``[..., K]``, w ``[N, K]``,
    bias ``[N]``, all bf16; N and K multiples of 16.

    The forward pass quantizes the weight (one pass, both orientations) and
    keeps the activations as the 8-bit checkpoint its GEMM reads.  Backward:
    ``dx = deq(q(dy)) @ deq(q(w))``, dy quantized like activations;
    ``dw = dy^T @ deq(q(x))`` and ``db`` from bf16 dy.  The quantizations
    are passed straight through.  Where no gradient can be asked for
    (torch.no_grad, or no operand requires one) nothing is kept.  A bias
    gradient alone keeps and computes what the weight's would.

    A step can be captured into a graph, after a warm-up on a side stream whose
    outputs may stay alive.  The backward pass of one is refused where a leaf's
    gradient accumulator is of the default stream, which no capture takes in:
    while an autograd graph of that leaf from there is alive, or something
    else holds it (a data-parallel wrapper: make it on the side stream).  So is
    one that another operator made first, on a stream not known here: until a
    backward() runs it on a side stream, or, in the capture itself, unless this
    operator is the first to be given the leaf.  Reverse mode only."""
    for t, name in ((x, "x"), (w, "w")) + (((bias, "bias"),) if bias is not None else ()):
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
        _require_cuda(t, name)
    if w.dim() != 2 or x.shape[-1] != w.shape[1] or w.shape[0] % 16 or w.shape[1] % 16:
        raise ValueError(f"x [..., K] and w [N, K] with N and K multiples of 16, got {tuple(x.shape)}, {tuple(w.shape)}")
    _same_device(x, w, bias)
    if not torch.is_grad_enabled() or not (x.requires_grad or w.requires_grad or
                                           (bias is not None and bias.requires_grad)):
        _reverse_only("linear_b128", x, w, bias)
        return _linear_b128_forward(x, w, bias, 0)[0]
    stream = _stream(x.device)
    _mark_leaves_before((x, w, bias), stream)
    y = _LinearB128.apply(x, w, bias)
    _mark_leaves(y, stream)
    return y


# ---------------------------------------------------------------------------
# MXFP4 on both sides
# ---------------------------------------------------------------------------

def mxfp8_linear_w4a4_workspace_bytes(M, N, K):
    return _bytes("mxfp8_linear_w4a4_workspace_bytes", M, N, K)


def mxfp8_linear_w4a4(x, M, K, ldx, wp, sp, N, bias, y, ldy, ws, ws_bytes, stream):
    return lib().mxfp8_linear_w4a4(x, M, K, ldx, wp, sp, N, bias, y, ldy, ws, ws_bytes, stream)


def mxfp8_debug_force_w4a4(form):
    _bytes.cache_clear()
    return lib().mxfp8_debug_force_w4a4(form)


class PackedActivationFP4(PackedActivation):
    """Activations quantized to MXFP4 in the packed operand layout (rows
    padded to 128): the activations of ``gemm_packed`` with a
    PreparedWeightFP4."""

    def dequantize(self):
        raise NotImplementedError("MXFP4 activations have no dequantize entry")

    def unpack(self):
        """(E2M1 ``[M_pad, K/2]``, two codes per byte, UE8M0 ``[M_pad, K/32]``)
        as uint8 tensors."""
        if self.M == 0:
            return self.q_packed.view(0, self.K // 2), self.s_packed.view(0, self.K // 32)
        with _on(self.device):
            return PreparedWeightFP4(self.q_packed, self.s_packed, self.M, self.K).unpack()


def quantize_act_packed_fp4(x):
    """bf16 ``x[..., K]`` (GPU, K % 256 == 0) -> PackedActivationFP4 (the rule
    of ``quantize_fp4``; a block with an infinity or a NaN gets the scale
    byte 0xFF, NaN)."""
    x2 = _rows(x, "x")
    M, K = x2.shape
    q, s = _sz(), _sz()
    _check(lib().mxfp8_packed_act_fp4_bytes(max(M, 1), K, ctypes.byref(q), ctypes.byref(s)),
           "mxfp8_packed_act_fp4_bytes")
    with _on(x.device):
        qp = x2.new_empty(q.value if M else 0, dtype=torch.uint8)
        sp = x2.new_empty(s.value if M else 0, dtype=torch.uint8)
        _check(lib().mxfp8_quantize_act_packed_fp4(_ptr(x2), M, K, x2.stride(0), _ptr(qp), _ptr(sp),
                                                   _stream(x.device)), "mxfp8_quantize_act_packed_fp4")
    return PackedActivationFP4(qp, sp, M, K)


def linear_w4a4(x, pw, bias=None, out=None):
    """The linear layer with MXFP4 on both sides: ``y = bf16(deq4(q4(x)) @
    deq4(W).T + bias)``, x bf16 ``[..., K]`` quantized to MXFP4 on the fly, pw
    a PreparedWeightFP4 (the weight ``linear`` multiplies with 8-bit
    activations), bias bf16 ``[N]`` or None.  Returns bf16 ``[..., N]``; ``out``:
    bf16 ``[M, N]`` to write into, M the rows of x, not overlapping x.  No
    gradients."""
    if not isinstance(pw, PreparedWeightFP4):
        raise ValueError("linear_w4a4 takes an MXFP4 weight (prepare_weight_fp4)")
    x2 = _rows(x, "x")
    (M, K), N = x2.shape, pw.N
    if K != pw.K:
        raise ValueError(f"x has {K} columns, the weight {pw.K}")
    bias = _bias(bias, N, align=4)
    if out is None:
        y = x.new_empty(M, N) if x.dim() == 2 else x.new_empty(*x.shape[:-1], N)
        ldy = N
    else:
        if out.dtype != torch.bfloat16 or tuple(out.shape) != (M, N) or out.stride(1) != 1 or out.stride(0) < N:
            raise ValueError(f"out must be bfloat16 [{M}, {N}] with contiguous rows that do not overlap")
        y, ldy = out, out.stride(0)
    _same_device(x2, pw.w_packed, bias, y)
    with _on(x.device):
        need = _bytes("mxfp8_linear_w4a4_workspace_bytes", M, N, K)
        ws = _scratch(need, x2)
        _check(lib().mxfp8_linear_w4a4(_ptr(x2), M, K, x2.stride(0), _ptr(pw.w_packed), _ptr(pw.s_packed), N,
                                       _ptr(bias), _ptr(y), ldy, _ptr(ws), need, _stream(x.device)),
               "mxfp8_linear_w4a4")
    return y if out is None or x.dim() == 2 else y.view(*x.shape[:-1], N)


# ---------------------------------------------------------------------------
# Routed MoE
# ---------------------------------------------------------------------------

def mxfp8_moe_prepared_bytes(E, H, I):
    out = [_sz() for _ in range(4)]
    _check(lib().mxfp8_moe_prepared_bytes(E, H, I, *[ctypes.byref(o) for o in out]), "mxfp8_moe_prepared_bytes")
    return tuple(o.value for o in out)


def mxfp8_moe_prepare_weights(w13, s13, w2, s2, E, H, I, w13p, s13p, w2p, s2p, stream):
    return lib().mxfp8_moe_prepare_weights(w13, s13, w2, s2, E, H, I, w13p, s13p, w2p, s2p, stream)


def mxfp8_moe_workspace_bytes(T, H, I, E, topk):
    b = _sz()
    _check(lib().mxfp8_moe_workspace_bytes(T, H, I, E, topk, ctypes.byref(b)), "mxfp8_moe_workspace_bytes")
    return b.value


def mxfp8_moe_grouped(x, logits, T, H, E, topk, I, w13p, s13p, w2p, s2p, y, ws, ws_bytes, stream):
    return lib().mxfp8_moe_grouped(x, logits, T, H, E, topk, I, w13p, s13p, w2p, s2p, y, ws, ws_bytes, stream)


def mxfp8_moe_debug_capture(act, q, s, ids, wts):
    return lib().mxfp8_moe_debug_capture(act, q, s, ids, wts)


class MoEWeights:
    """Expert weights after the one-time preparation (opaque packed layouts)."""

    def __init__(self, w13p, s13p, w2p, s2p, E, H, I):
        self.w13p, self.s13p, self.w2p, self.s2p = w13p, s13p, w2p, s2p
        self.E, self.H, self.I = E, H, I

    @property
    def device(self):
        return self.w13p.device


def moe_prepare_weights(w13_q, w13_s, w2_q, w2_s):
    """MXFP8 expert weights -> MoEWeights.

    ``w13_q`` E4M3 ``[E, 2I, H]`` (gate rows then up rows) with UE8M0 ``w13_s``
    ``[E, 2I, H/32]``; ``w2_q`` ``[E, H, I]`` with ``w2_s`` ``[E, H, I/32]``
    (uint8 or float8_e4m3fn, GPU)."""
    w13_q, w13_s, w2_q, w2_s = (_as_bytes(t).contiguous() for t in (w13_q, w13_s, w2_q, w2_s))
    _require_cuda(w13_q, "w13_q")
    E, two_i, H = w13_q.shape
    I = two_i // 2
    assert w2_q.shape == (E, H, I) and w13_s.shape == (E, 2 * I, H // 32) and w2_s.shape == (E, H, I // 32)
    b = mxfp8_moe_prepared_bytes(E, H, I)
    outs = [torch.empty(n, dtype=torch.uint8, device=w13_q.device) for n in b]
    _check(mxfp8_moe_prepare_weights(_ptr(w13_q), _ptr(w13_s), _ptr(w2_q), _ptr(w2_s), E, H, I,
                                     *[_ptr(o) for o in outs], _stream(w13_q.device)), "mxfp8_moe_prepare_weights")
    return MoEWeights(*outs, E, H, I)


_moe_workspaces = {}


def moe_workspace(T, H, I, E, topk, device):
    """The MoE layer's workspace, cached per (device, current stream) like
    ``workspace`` (superseded buffers are kept, never freed)."""
    return _workspace_sized(mxfp8_moe_workspace_bytes(T, H, I, E, topk), device, cache=_moe_workspaces, zero=False)


def moe_grouped(x, logits, mw, topk, out=None):
    """The MXFP8 routed MoE layer: ``x`` bf16 ``[T, H]``, ``logits`` fp32
    ``[T, E]``, ``mw`` MoEWeights -> bf16 ``[T, H]``."""
    assert x.dtype == torch.bfloat16, f"MXFP8 MoE takes bfloat16 activations, got {x.dtype}"
    assert logits.dtype == torch.float32
    _require_cuda(x, "x")
    x = x.contiguous()
    logits = logits.contiguous()
    T, H = x.shape
    assert H == mw.H and logits.shape == (T, mw.E)
    y = out if out is not None else torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    ws = moe_workspace(T, H, mw.I, mw.E, topk, x.device)
    _check(mxfp8_moe_grouped(_ptr(x), _ptr(logits), T, H, mw.E, topk, mw.I, _ptr(mw.w13p), _ptr(mw.s13p),
                             _ptr(mw.w2p), _ptr(mw.s2p), _ptr(y), _ptr(ws), ws.numel(), _stream(x.device)),
           "mxfp8_moe_grouped")
    return y


def moe_debug_capture(act=None, q=None, s=None, ids=None, wts=None):
    """Test hook: capture, per row t*k + j, the gated activation (bf16
    ``[T*k, I]``), its MX quantization (``[T*k, I]`` / ``[T*k, I/32]`` uint8),
    the routed expert (int32 ``[T*k]``) and routing weight (fp32 ``[T*k]``) of
    later MoE calls; no arguments turns it off."""
    _check(mxfp8_moe_debug_capture(_ptr(act), _ptr(q), _ptr(s), _ptr(ids), _ptr(wts)), "mxfp8_moe_debug_capture")


def _router_args(logits, valid):
    if logits.dtype not in _DTYPES or logits.dim() != 2:
        raise ValueError(f"logits must be float32 or bfloat16 [T, E], got {logits.dtype} {tuple(logits.shape)}")
    _require_cuda(logits, "logits")
    if logits.stride(-1) != 1 or logits.stride(0) < logits.shape[1]:
        logits = logits.clone(memory_format=torch.contiguous_format)
    if valid is not None:
        if valid.dtype not in (torch.bool, torch.uint8) or tuple(valid.shape) != (logits.shape[0],):
            raise ValueError(f"valid must be bool or uint8 [{logits.shape[0]}]")
        valid = valid.contiguous()
        _same_device(logits, valid)
    return logits, valid


def moe_balance(logits, topk, valid=None, coef=1e-2, z_coef=0.0):
    """Load-balance and z loss of the router of ``moe_grouped``: ``(loss,
    counts, used)``, fp32 scalar, int32 ``[E]`` tokens of each expert, int32
    ``[1]`` tokens counted.

    ``loss = coef E / (topk n^2) sum_e counts[e] sum_t softmax(logits)[t, e] +
    z_coef / n sum_t logsumexp(logits[t])^2`` over the n tokens with ``valid``
    set and a logit other than -inf.  ``logits`` ``[T, E]`` fp32 or bf16; the
    gradient is ``moe_balance_backward``'s (``moe_balance_loss`` for autograd)."""
    logits, valid = _router_args(logits, valid)
    T, E = logits.shape
    d = logits.device
    with _on(d):
        loss = logits.new_empty((), dtype=torch.float32)
        counts = logits.new_empty(E, dtype=torch.int32)
        used = logits.new_empty(1, dtype=torch.int32)
        need = _bytes("mxfp8_moe_balance_workspace_bytes", T, E)
        ws = _scratch(need, counts)
        _check(lib().mxfp8_moe_balance(_ptr(logits), _DTYPES[logits.dtype], T, E, logits.stride(0), topk,
                                       _ptr(valid), coef, z_coef, _ptr(loss), _ptr(counts), _ptr(used), _ptr(ws),
                                       need, _stream(d)), "mxfp8_moe_balance")
    return loss, counts, used


def moe_balance_backward(logits, topk, counts, used, valid=None, coef=1e-2, z_coef=0.0, grad=None):
    """Gradient of ``moe_balance``'s loss with respect to the logits (their
    shape and type), counts held constant.  ``counts`` and ``used`` as
    ``moe_balance`` returned them, or summed over data-parallel ranks;
    ``grad``: fp32 GPU scalar that multiplies it (None: 1)."""
    logits, valid = _router_args(logits, valid)
    T, E = logits.shape
    if counts.dtype != torch.int32 or counts.shape != (E,) or used.dtype != torch.int32 or used.numel() != 1:
        raise ValueError(f"counts must be int32 [{E}] and used int32 [1]")
    if grad is not None and (grad.dtype != torch.float32 or grad.numel() != 1):
        raise ValueError("grad must be one float32")
    counts = counts.contiguous()
    _same_device(logits, counts, used, grad)
    with _on(logits.device):
        d = logits.new_empty(T, E)
        _check(lib().mxfp8_moe_balance_backward(_ptr(logits), _DTYPES[logits.dtype], T, E, logits.stride(0), topk,
                                                _ptr(valid), coef, z_coef, _ptr(counts), _ptr(used), _ptr(grad),
                                                _ptr(d), E, _stream(logits.device)), "mxfp8_moe_balance_backward")
    return d


class _MoEBalance(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, topk, valid, coef, z_coef):
        loss, counts, used = moe_balance(logits, topk, valid, coef, z_coef)
        ctx.save_for_backward(logits, counts, used, valid)
        ctx.args = topk, coef, z_coef
        if ctx.needs_input_grad[0]:
            # The caller gets counts of its own: a collective over ranks writes
            # into them without autograd's notice, and the gradient needs the
            # ones that go with this call's tokens.  (A kernel, not a copy: it
            # may be captured.)
            counts = counts + 0
        ctx.mark_non_differentiable(counts)
        return loss, counts

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, _):
        _check_capture(ctx, _stream(grad.device), torch.cuda.is_current_stream_capturing())
        logits, counts, used, valid = ctx.saved_tensors
        topk, coef, z_coef = ctx.args
        return moe_balance_backward(logits, topk, counts, used, valid, coef, z_coef, grad), None, None, None, None


def moe_balance_loss(logits, topk, valid=None, coef=1e-2, z_coef=0.0):
    """``moe_balance`` for autograd: ``(loss, counts)``, the loss
    differentiable with respect to ``logits``.  ``counts`` are the caller's to
    change (an all-reduce over ranks, say): the gradient does not read them.
    In captured graphs, and in reverse mode only, as ``linear_b128``."""
    stream = _stream(logits.device) if logits.is_cuda else _LEGACY   # (moe_balance refuses the others)
    if torch.is_grad_enabled():
        _mark_leaves_before((logits,), stream)
    loss, counts = _MoEBalance.apply(logits, topk, valid, coef, z_coef)
    if loss.requires_grad:
        _mark_leaves(loss, stream)
    return loss, counts


# ---------------------------------------------------------------------------
# Tokens sorted by expert and back, and the experts' MXFP4 products
# ---------------------------------------------------------------------------

class MoEOrder:
    """The slots of T tokens (``topk`` each) sorted by expert.

    ``rows`` int32 ``[T, topk]``: the sorted row of each slot, by expert and
    within one by slot; slots without an expert come behind all others.
    ``slots`` int32 ``[T * topk]``: the slot of each row.  ``offsets`` int32
    ``[E + 1]``: the first row of each expert, and the number of rows that have
    one.  All contiguous and on one device.  ``moe_sort`` makes it; built from
    tensors of one's own these are checked, but what they hold is not (values
    that no sort gives make wrong or unwritten rows)."""

    def __init__(self, rows, slots, offsets):
        for t, name, dim in ((rows, "rows", 2), (slots, "slots", 1), (offsets, "offsets", 1)):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.dim() != dim or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous int32 with {dim} dimension{'s'[:dim - 1]}")
        if slots.numel() != rows.numel() or offsets.numel() < 2:
            raise ValueError(f"slots must be int32 [{rows.numel()}] and offsets int32 [E + 1], got {slots.numel()} and "
                             f"{offsets.numel()}")
        if not rows.device == slots.device == offsets.device:
            raise ValueError(f"operands on {rows.device}, {slots.device} and {offsets.device}")
        self.rows, self.slots, self.offsets = rows, slots, offsets
        self.T, self.topk = rows.shape
        self.E = offsets.numel() - 1

    @classmethod
    def _of(cls, rows, slots, offsets, T, topk, E):
        """Of tensors made here, without the checks."""
        order = cls.__new__(cls)
        order.rows, order.slots, order.offsets = rows, slots, offsets
        order.T, order.topk, order.E = T, topk, E
        return order

    @property
    def _kept(self):
        """Address of the number of rows with an expert."""
        return self.offsets.data_ptr() + 4 * self.E

    @property
    def device(self):
        return self.rows.device


def moe_sort(ids, E):
    """Sorts the slots of a routed batch by their expert (stable): ``ids`` int32
    or int64 ``[T, topk]`` (``torch.topk``'s indices, say) over experts 0 .. E -
    1 -> MoEOrder.  Any other id (-1 for padding, or an expert of another rank)
    is a slot without an expert here."""
    if ids.dtype not in (torch.int32, torch.int64) or ids.dim() != 2:
        raise ValueError(f"ids must be int32 or int64 [T, topk], got {ids.dtype} {tuple(ids.shape)}")
    _require_cuda(ids, "ids")
    if not ids.is_contiguous():
        ids = ids.contiguous()
    T, topk = ids.shape
    if not 1 <= topk <= 16:
        raise ValueError(f"topk must be 1 to 16, got {topk}")
    R = T * topk
    with _on(ids.device):
        rows = ids.new_empty(T, topk, dtype=torch.int32)
        slots = ids.new_empty(R, dtype=torch.int32)
        need = _bytes("mxfp8_moe_sort_workspace_bytes", R, E)
        offsets = ids.new_empty(E + 1, dtype=torch.int32)
        ws = _scratch(need, ids)
        _check(lib().mxfp8_moe_sort(_ptr(ids), ids.element_size(), R, E, _ptr(rows), _ptr(slots), _ptr(offsets),
                                    _ptr(ws), need, _stream(ids.device)), "mxfp8_moe_sort")
    return MoEOrder._of(rows, slots, offsets, T, topk, E)


def _matrix(x, rows, name):
    """Checks that x is fp32 or bf16 ``[rows, H]`` on the GPU."""
    if x.dtype not in _DTYPES or x.dim() != 2 or x.shape[0] != rows:
        raise ValueError(f"{name} must be float32 or bfloat16 [{rows}, H], got {x.dtype} {tuple(x.shape)}")
    _require_cuda(x, name)


def _laid_out(x):
    """x with contiguous rows that do not overlap.  Called inside of the autograd
    nodes: a copy made before them would be a node of its own, and hide its
    leaf from ``_mark_leaves`` and ``_check_capture``."""
    row, col = x.stride()
    if col != 1 or row < x.shape[1]:
        x = x.clone(memory_format=torch.contiguous_format)
    return x


def _require_order(order):
    if not isinstance(order, MoEOrder):
        raise ValueError("order must be a MoEOrder (moe_sort)")


def _permute(x, order):
    H, R = x.shape[1], order.T * order.topk
    with _on(x.device):
        xs = x.new_empty(R, H)
        _check(lib().mxfp8_moe_permute(_ptr(x), _DTYPES[x.dtype], order.T, H, x.stride(0), order.topk,
                                       _ptr(order.rows), order._kept, _ptr(xs), H, _stream(x.device)),
               "mxfp8_moe_permute")
    return xs


def _unpermute(ys, order, weights):
    H = ys.shape[1]
    with _on(ys.device):
        y = ys.new_empty(order.T, H)
        _check(lib().mxfp8_moe_unpermute(_ptr(ys), _DTYPES[ys.dtype], order.T, H, ys.stride(0), order.topk,
                                         _ptr(order.rows), order._kept, _ptr(weights), _ptr(y), H,
                                         _stream(ys.device)), "mxfp8_moe_unpermute")
    return y


def _backward_once(backward):
    """``backward`` for a Function whose gradient has none of its own: torch's
    wrapper, which makes second derivatives an error, costs some microseconds
    and changes nothing in an ordinary pass."""
    once = torch.autograd.function.once_differentiable(backward)
    return staticmethod(lambda ctx, d: once(ctx, d) if torch.is_grad_enabled() else backward(ctx, d))


def _keep_order(ctx, order):
    """Keeps an order for the backward pass.  (Not by save_for_backward: permute's
    gradient needs no retained graph for a second pass.)"""
    rows, offsets = order.rows, order.offsets
    try:
        version = rows._version + offsets._version
    except RuntimeError:                           # inference tensors have none
        version = None
    ctx.kept = order, rows, offsets, version


def _kept_order(ctx):
    order, rows, offsets, version = ctx.kept
    if order.rows is not rows or order.offsets is not offsets or \
            (version is not None and rows._version + offsets._version != version):
        raise RuntimeError("the rows or offsets of an order have been modified by an inplace operation or replaced "
                           "between the forward and the backward pass")
    return order


class _MoEPermute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, order):
        _keep_order(ctx, order)
        return _permute(_laid_out(x), order)

    @_backward_once
    def backward(ctx, dxs):
        if torch.cuda.is_current_stream_capturing():
            _check_capture(ctx, _stream(dxs.device), True)
        return _unpermute(_laid_out(dxs), _kept_order(ctx), None), None


class _MoEUnpermute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, weights, order):
        _keep_order(ctx, order)
        ys = _laid_out(ys)
        if weights is not None and not weights.is_contiguous():
            weights = weights.contiguous()
        ctx.save_for_backward(ys if ctx.needs_input_grad[1] else None, weights)
        return _unpermute(ys, order, weights)

    @_backward_once
    def backward(ctx, dy):
        stream = _stream(dy.device)
        if torch.cuda.is_current_stream_capturing():
            _check_capture(ctx, stream, True)
        need_ys, need_w, _ = ctx.needs_input_grad
        ys, weights = ctx.saved_tensors
        order = _kept_order(ctx)
        dy = _laid_out(dy)
        H = dy.shape[1]
        with _on(dy.device):
            dys = dy.new_empty(order.T * order.topk, H) if need_ys else None
            dw = dy.new_empty(order.T, order.topk, dtype=torch.float32) if need_w else None
            _check(lib().mxfp8_moe_unpermute_backward(_ptr(dy), _DTYPES[dy.dtype], order.T, H, dy.stride(0), order.topk,
                                                      _ptr(order.rows), order._kept, _ptr(ys),
                                                      0 if ys is None else ys.stride(0), _ptr(weights), _ptr(dys), H,
                                                      _ptr(dw), stream), "mxfp8_moe_unpermute_backward")
        return dys, dw, None


def moe_permute(x, order):
    """The rows of ``x`` fp32 or bf16 ``[T, H]`` in the order of their experts:
    ``xs[order.rows[t, j]] = x[t]``, ``[T * topk, H]``, zeros in the rows of
    slots without an expert.  Differentiable; the gradient adds a token's rows
    in fp32, in slot order.  In captured graphs, and in reverse mode only, as
    ``linear_b128``."""
    _require_order(order)
    _matrix(x, order.T, "x")
    _same_device(x, order.rows)
    if not (torch.is_grad_enabled() and x.requires_grad):
        _reverse_only("moe_permute", x)
        return _permute(_laid_out(x), order)
    stream = _stream(x.device)
    _mark_leaves_before((x,), stream)
    xs = _MoEPermute.apply(x, order)
    _mark_leaves(xs, stream)
    return xs


def moe_unpermute(ys, order, weights=None):
    """The experts' rows back with their tokens: ``y[t] = sum_j weights[t, j]
    ys[order.rows[t, j]]`` over the slots with an expert, ``ys`` fp32 or bf16
    ``[T * topk, H]`` -> ``[T, H]``, summed in fp32 in slot order and rounded
    once.  ``weights`` fp32 ``[T, topk]``, or None for all 1.  Differentiable
    with respect to ys and weights (0 for slots without an expert).  In captured
    graphs, and in reverse mode only, as ``linear_b128``."""
    _require_order(order)
    _matrix(ys, order.T * order.topk, "ys")
    if weights is not None and (weights.dtype != torch.float32 or weights.shape != order.rows.shape):
        raise ValueError(f"weights must be float32 [{order.T}, {order.topk}]")
    _same_device(ys, order.rows, weights)
    if not torch.is_grad_enabled() or not (ys.requires_grad or (weights is not None and weights.requires_grad)):
        _reverse_only("moe_unpermute", ys, weights)
        return _unpermute(_laid_out(ys), order, None if weights is None else weights.contiguous())
    stream = _stream(ys.device)
    _mark_leaves_before((ys, weights), stream)
    y = _MoEUnpermute.apply(ys, weights, order)
    _mark_leaves(y, stream)
    return y


class ExpertWeightsFP4:
    """The experts' MXFP4 weights ``[E, N, K]`` after the one-time preparation
    (opaque packed layout)."""

    def __init__(self, w_packed, s_packed, E, N, K):
        self.w_packed, self.s_packed = w_packed, s_packed
        self.E, self.N, self.K = E, N, K

    @property
    def device(self):
        return self.w_packed.device


def moe_prepare_experts_fp4(w_e2m1, w_s):
    """MXFP4 expert weights ``w_e2m1`` uint8 ``[E, N, K/2]`` (two E2M1 codes per
    byte, element 2j in the low nibble) with UE8M0 scales ``w_s`` ``[E, N,
    K/32]`` -> ExpertWeightsFP4."""
    w, s = _as_bytes(w_e2m1).contiguous(), _as_bytes(w_s).contiguous()
    _require_cuda(w, "w_e2m1")
    if w.dim() != 3 or tuple(s.shape) != (w.shape[0], w.shape[1], w.shape[2] // 16):
        raise ValueError(f"w_e2m1 [E, N, K/2] and w_s [E, N, K/32], got {tuple(w.shape)}, {tuple(s.shape)}")
    _same_device(w, s)
    if w.data_ptr() % 16 != 0:
        w = w.clone()
    E, N, K = w.shape[0], w.shape[1], 2 * w.shape[2]
    wb, sb = _sz(), _sz()
    _check(lib().mxfp8_moe_prepared_experts_fp4_bytes(E, N, K, ctypes.byref(wb), ctypes.byref(sb)),
           "mxfp8_moe_prepared_experts_fp4_bytes")
    with _on(w.device):
        wp, sp = w.new_empty(wb.value), w.new_empty(sb.value)
        _check(lib().mxfp8_moe_prepare_experts_fp4(_ptr(w), _ptr(s), E, N, K, _ptr(wp), _ptr(sp), _stream(w.device)),
               "mxfp8_moe_prepare_experts_fp4")
    return ExpertWeightsFP4(wp, sp, E, N, K)


def moe_linear_w4a4(x, ew, order, gather=False):
    """The experts' products on sorted rows, MXFP4 on both sides: ``y[r] =
    bf16(deq4(q4(x[r])) @ deq4(W[e(r)]).T)``, e(r) the expert of row r; zeros in
    the rows of slots without an expert.

    ``x`` bf16 ``[T * topk, K]`` in ``order``'s rows or, with ``gather``, ``[T, K]``:
    the tokens, each row r taking its own (``moe_permute(x)`` without the copy).
    ``ew`` ExpertWeightsFP4.  Returns bf16 ``[T * topk, N]``.  No gradients."""
    _require_order(order)
    if not isinstance(ew, ExpertWeightsFP4):
        raise ValueError("ew must be ExpertWeightsFP4 (moe_prepare_experts_fp4)")
    R = order.T * order.topk
    if x.dim() != 2 or x.shape[0] != (order.T if gather else R) or x.shape[1] != ew.K or order.E != ew.E:
        raise ValueError(f"x [{order.T if gather else R}, {ew.K}] and an order over {ew.E} experts, got "
                         f"{tuple(x.shape)} and {order.E}")
    x = _rows(x, "x")
    _same_device(x, ew.w_packed, order.rows)
    with _on(x.device):
        y = x.new_empty(R, ew.N)
        need = _bytes("mxfp8_moe_linear_w4a4_workspace_bytes", x.shape[0], R, ew.N, ew.K, ew.E)
        ws = _scratch(need, x)
        _check(lib().mxfp8_moe_linear_w4a4(_ptr(x), x.shape[0], ew.K, x.stride(0), _ptr(order.slots) if gather else None,
                                           order.topk, _ptr(order.offsets), R, ew.E, _ptr(ew.w_packed),
                                           _ptr(ew.s_packed), ew.N, _ptr(y), ew.N, _ptr(ws), need, _stream(x.device)),
               "mxfp8_moe_linear_w4a4")
    return y
