"""Thin Python binding of ``libsq.so`` (include/sq.h).

Argument marshalling only: every call checks the tensors it is given, turns
them into device pointers and sizes, and calls the C ABI on the current torch
CUDA stream.  Output tensors are allocated here with torch when the caller
does not pass them; the library itself never allocates.  There is no CPU or
PyTorch fallback: if the library is missing or a call fails, an exception is
raised.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from . import build as _build

SQ_OK = 0
STATUS_NAMES = {
    0: "SQ_OK", 1: "SQ_ERR_INVALID_ARG", 2: "SQ_ERR_UNSUPPORTED", 3: "SQ_ERR_ALIGNMENT",
    4: "SQ_ERR_OVERFLOW_RISK", 5: "SQ_ERR_CUDA", 6: "SQ_ERR_PIPELINE_TIMEOUT",
    7: "SQ_ERR_WORKSPACE",
}
SQ_F32, SQ_BF16 = 0, 1
NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
EPI = {"bf16": 0, "bf16_relu": 1, "i32": 2, "f32": 3}
MAX_K = 133144

# Every symbol include/sq.h declares.
EXPORTS = (
    "sq_calibrate_absmax", "sq_compute_smooth_scales", "sq_smooth_quantize_weights",
    "sq_norm_smooth_quant_per_token", "sq_w8a8_gemm_workspace_size", "sq_w8a8_gemm_dequant",
    "sq_linear_w8a8", "sq_status_string", "sq_get_device_error", "sq_set_wait_limit",
    "sq_w8a8_gemm_dequant_noalloc", "sq_w8a8_gemm_plan", "sq_norm_smooth_absmax",
    "sq_norm_smooth_quant_per_tensor", "sq_smooth_quantize_weights_per_tensor",
    "sq_w8a8_gemm_dequant_rowmax", "sq_quant_per_token_given_absmax",
    "sq_silu_mul_quant_per_token", "sq_norm_smooth_quant_per_token_fp8",
    "sq_smooth_quantize_weights_fp8", "sq_fp8_gemm_dequant", "sq_weight_column_max",
    "sq_smooth_scales_from_maxima", "sq_silu_mul_quant_per_token_fp8", "sq_row_absmax",
    "sq_dequant_i32", "sq_llmint8_outliers", "sq_llmint8_combine",
    "sq_moe_route_workspace_size", "sq_moe_route", "sq_w8a8_gemm_grouped", "sq_fp8_gemm_grouped",
    "sq_block_norm_quant_per_token", "sq_block_norm_quant_per_token_fp8",
)
LLMINT8_MAX_K = 1 << 20
NOALLOC_SCRATCH_BYTES = 8 << 20
MOE_MAX_EXPERTS, MOE_MAX_TOP_K = 512, 16
MOE_SCORES = {"softmax": 0, "sigmoid": 1}
BLOCK_NORM_MAX_K = 32768


class GemmPlanInfo(ctypes.Structure):
    """sq_gemm_plan_info: what sq_w8a8_gemm_dequant runs for a shape."""
    _fields_ = [("kernel", ctypes.c_int), ("tile_m", ctypes.c_int), ("tile_n", ctypes.c_int),
                ("split_k", ctypes.c_int), ("stream_k", ctypes.c_int), ("ctas", ctypes.c_int),
                ("launches", ctypes.c_int), ("workspace_bytes", ctypes.c_size_t)]

    KERNELS = ("w8a8_gemm_kernel", "w8a8_gemm_pair_kernel", "w8a8_gemm_kernel (decode tiles)")

    def as_dict(self):
        d = {f: getattr(self, f) for f, _ in self._fields_}
        d["kernel_name"] = self.KERNELS[self.kernel]
        return d


class BlockNormArgs(ctypes.Structure):
    """sq_block_norm_args: the arguments of sq_block_norm_quant_per_token."""
    _fields_ = [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("R", ctypes.c_int64),
                ("token_row", ctypes.c_void_p), ("weights", ctypes.c_void_p),
                ("top_k", ctypes.c_int), ("dtype", ctypes.c_int), ("M", ctypes.c_int64),
                ("K", ctypes.c_int64), ("post_norm", ctypes.c_int),
                ("post_gamma", ctypes.c_void_p), ("post_beta", ctypes.c_void_p),
                ("post_eps", ctypes.c_float), ("gate", ctypes.c_void_p),
                ("token_gate", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("ld_res", ctypes.c_int64), ("residual_scale", ctypes.c_float),
                ("pre_norm", ctypes.c_int), ("pre_gamma", ctypes.c_void_p),
                ("pre_beta", ctypes.c_void_p), ("pre_eps", ctypes.c_float),
                ("h_out", ctypes.c_void_p), ("ld_h", ctypes.c_int64), ("Xq", ctypes.c_void_p),
                ("x_scale", ctypes.c_void_p)]


class SQError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__("%s failed: %s" % (call, _status_text(status)))


_lib: Optional[ctypes.CDLL] = None


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """Load libsq.so (built in-tree); raises if it is not there."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError("libsq.so is not built (%s); run python -m "
                               "w8a8_int8_quantized_norm_b200.build" % path)
        L = ctypes.CDLL(path)
        _declare(L)
        _lib = L
    return _lib


_P, _I64, _I32, _F32, _F64, _SZ = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                                   ctypes.c_double, ctypes.c_size_t)


def _declare(L):
    L.sq_calibrate_absmax.argtypes = [_P, _I32, _I64, _I64, _I64, _I32, _P, _P, _F32, _P, _P]
    L.sq_compute_smooth_scales.argtypes = [_P, _P, _P, _I32, _I32, _I64, _F64, _F32, _P, _P, _P,
                                           _P, _P, _P]
    L.sq_smooth_quantize_weights.argtypes = [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _P]
    L.sq_norm_smooth_quant_per_token.argtypes = [_P, _I32, _I64, _I64, _I64, _I32, _P, _P, _F32,
                                                 _P, _P, _P]
    L.sq_w8a8_gemm_workspace_size.argtypes = [_I64, _I64, _I64, _I32]
    L.sq_w8a8_gemm_workspace_size.restype = _SZ
    L.sq_w8a8_gemm_dequant.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _I64, _P, _SZ,
                                       _I32, _I32, _P]
    L.sq_w8a8_gemm_dequant_noalloc.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _I64,
                                               _I32, _I32, _P]
    L.sq_linear_w8a8.argtypes = [_P, _I32, _I64, _I64, _I64, _I32, _P, _P, _F32, _P, _P, _I64,
                                 _I32, _P, _I64, _P, _P, _P, _SZ, _P]
    L.sq_status_string.argtypes = [_I32]
    L.sq_status_string.restype = ctypes.c_char_p
    L.sq_get_device_error.argtypes = [_P]
    L.sq_norm_smooth_absmax.argtypes = [_P, _I32, _I64, _I64, _I64, _I32, _P, _P, _F32, _P, _P]
    L.sq_norm_smooth_quant_per_tensor.argtypes = [_P, _I32, _I64, _I64, _I64, _I32, _P, _P, _F32,
                                                  _P, _P, _P, _P]
    L.sq_smooth_quantize_weights_per_tensor.argtypes = [_P, _I32, _I64, _I64, _I64, _P, _P, _P,
                                                        _P, _P]
    L.sq_w8a8_gemm_dequant_rowmax.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _I64,
                                              _P, _I32, _P]
    L.sq_quant_per_token_given_absmax.argtypes = [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _P]
    L.sq_row_absmax.argtypes = [_P, _I32, _I64, _I64, _I64, _P, _P]
    L.sq_llmint8_outliers.argtypes = [_P, _I64, _F32, _P, _P, _P, _P]
    L.sq_llmint8_combine.argtypes = [_P, _I64, _I64, _I64, _P, _P, _P, _I32, _I64, _P, _I32,
                                     _I64, _I64, _P, _P, _I32, _P, _I64, _P]
    L.sq_dequant_i32.argtypes = [_P, _I64, _I64, _I64, _P, _P, _I32, _P, _I64, _P]
    L.sq_silu_mul_quant_per_token.argtypes = [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _I64, _P]
    L.sq_norm_smooth_quant_per_token_fp8.argtypes = [_P, _I32, _I64, _I64, _I64, _I32, _P, _P,
                                                     _F32, _P, _P, _P]
    L.sq_smooth_quantize_weights_fp8.argtypes = [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _P]
    L.sq_fp8_gemm_dequant.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _I64, _P, _SZ,
                                      _I32, _P]
    L.sq_silu_mul_quant_per_token_fp8.argtypes = [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _I64,
                                                  _P]
    L.sq_weight_column_max.argtypes = [_P, _P, _I32, _I32, _I64, _P, _P]
    L.sq_smooth_scales_from_maxima.argtypes = [_P, _P, _I64, _F64, _F32, _P, _P, _P, _P, _P, _P]
    L.sq_w8a8_gemm_plan.argtypes = [_I64, _I64, _I64, _I32, _I32, ctypes.POINTER(GemmPlanInfo)]
    L.sq_set_wait_limit.argtypes = [_I64]
    L.sq_set_wait_limit.restype = None
    L.sq_moe_route_workspace_size.argtypes = [_I64, _I64, _I32]
    L.sq_moe_route_workspace_size.restype = _SZ
    L.sq_moe_route.argtypes = [_P, _I32, _I64, _I64, _I64, _I32, _I32, _P, _I32, _F32, _P, _P, _P,
                               _P, _P, _P, _SZ, _P]
    L.sq_w8a8_gemm_grouped.argtypes = [_P, _I64, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I32,
                                       _P, _I64, _I32, _P]
    L.sq_fp8_gemm_grouped.argtypes = L.sq_w8a8_gemm_grouped.argtypes
    L.sq_block_norm_quant_per_token.argtypes = [ctypes.POINTER(BlockNormArgs), _P]
    L.sq_block_norm_quant_per_token_fp8.argtypes = [ctypes.POINTER(BlockNormArgs), _P]
    for name in EXPORTS:
        f = getattr(L, name)
        if f.argtypes is None:  # every call passes 64-bit sizes: no implicit int conversion
            raise RuntimeError("no argument types declared for %s" % name)
        if name not in ("sq_w8a8_gemm_workspace_size", "sq_status_string", "sq_set_wait_limit",
                        "sq_moe_route_workspace_size"):
            f.restype = _I32


def _status_text(status: int) -> str:
    try:
        return lib().sq_status_string(status).decode()
    except Exception:  # the library may be what failed to load
        return STATUS_NAMES.get(status, str(status))


def _check(status: int, call: str):
    if status != SQ_OK:
        raise SQError(status, call)


# The current stream's handle and the current device, without building the
# Python objects around them: a single-token call costs about as much host time
# as these do (3.2 us of torch.cuda.current_stream() against 0.1 us).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_get_stream = getattr(torch._C, "_cuda_getCurrentStream", None)
_set_stream = getattr(torch._C, "_cuda_setStream", None)
_NO_SCOPE = contextlib.nullcontext()


def _stream(stream=None):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    if torch.cuda.is_initialized():
        return ctypes.c_void_p(_raw_stream(_raw_device()))
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


class _OnStream:
    """torch.cuda.stream(stream) where the stream's device is current already: a
    call costs 2 us more in it, 8 us in the general one."""
    __slots__ = ("stream", "before")

    def __init__(self, stream):
        self.stream = stream

    def __enter__(self):
        s = self.stream
        self.before = _get_stream(s.device_index)
        _set_stream(stream_id=s.stream_id, device_index=s.device_index, device_type=s.device_type)

    def __exit__(self, *exc):
        i, index, kind = self.before
        _set_stream(stream_id=i, device_index=index, device_type=kind)


def _scope(device: torch.device, stream):
    """The context of a call on tensors of ``device``: that device current, and
    what the call allocates taken from the memory of the stream it runs on."""
    if device.type != "cuda":  # the call itself refuses such tensors
        return _NO_SCOPE
    if stream is not None:
        if stream.device != device:
            raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, device))
        if _raw_device() != device.index or _get_stream is None or _set_stream is None:
            return torch.cuda.stream(stream)
        return _OnStream(stream)
    return _NO_SCOPE if _raw_device() == device.index else torch.cuda.device(device)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SQ_BF16
    if t.dtype == torch.float32:
        return SQ_F32
    raise TypeError("activations and weights are bf16 or fp32, got %s" % t.dtype)


def _rows(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1 and t.shape[0] > 0):
        raise ValueError("%s must be 2-D with unit column stride" % name)
    # no row has no stride, and a single row's is arbitrary (numpy / torch may
    # report 0 for either)
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    return t.shape[0], t.shape[1], ld


def _vec(t: Optional[torch.Tensor], K: int, name: str):
    if t is None:
        return None
    if not (t.is_cuda and t.dtype == torch.float32 and t.dim() == 1 and t.numel() == K
            and t.is_contiguous()):
        raise ValueError("%s must be a contiguous fp32 CUDA vector of length %d" % (name, K))
    return t


# ---------------------------------------------------------------------------
# the six calls of the C ABI
# ---------------------------------------------------------------------------

def calibrate_absmax(x: torch.Tensor, norm: int, gamma=None, beta=None, eps: float = 1e-5,
                     act_max: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    M, K, ld = _rows(x, "x")
    with _scope(x.device, stream):
        if act_max is None:
            act_max = torch.zeros(K, dtype=torch.float32, device=x.device)
        _vec(act_max, K, "act_max")
        _check(lib().sq_calibrate_absmax(_ptr(x), _dtype_code(x), M, K, ld, norm,
                                         _ptr(_vec(gamma, K, "gamma")), _ptr(_vec(beta, K, "beta")),
                                         eps, _ptr(act_max), _stream(stream)),
               "sq_calibrate_absmax")
    return act_max


def compute_smooth_scales(act_max: torch.Tensor, weights: Sequence[torch.Tensor], alpha: float,
                          clamp_eps: float = 1e-5, gamma=None, beta=None, s=None,
                          gamma_folded=None, beta_folded=None, stream=None
                          ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    K = act_max.numel()
    _vec(act_max, K, "act_max")
    dt = _dtype_code(weights[0])
    for w in weights:
        _rows(w, "W")
        if not w.is_contiguous() or w.shape[1] != K or _dtype_code(w) != dt:
            raise ValueError("weights must be contiguous [N, K] of one dtype")
    ptrs = (ctypes.c_void_p * len(weights))(*[w.data_ptr() for w in weights])
    ns = (ctypes.c_int64 * len(weights))(*[w.shape[0] for w in weights])
    dev = act_max.device
    with _scope(dev, stream):
        s = torch.empty(K, dtype=torch.float32, device=dev) if s is None else _vec(s, K, "s")
        gf = (torch.empty(K, dtype=torch.float32, device=dev) if gamma_folded is None
              else _vec(gamma_folded, K, "gamma_folded"))
        bf = None
        if beta is not None:
            bf = (torch.empty(K, dtype=torch.float32, device=dev) if beta_folded is None
                  else _vec(beta_folded, K, "beta_folded"))
        _check(lib().sq_compute_smooth_scales(
            _ptr(act_max), ctypes.cast(ptrs, ctypes.c_void_p), ctypes.cast(ns, ctypes.c_void_p),
            len(weights), dt, K, float(alpha), clamp_eps, _ptr(_vec(gamma, K, "gamma")),
            _ptr(_vec(beta, K, "beta")), _ptr(s), _ptr(gf), _ptr(bf), _stream(stream)),
            "sq_compute_smooth_scales")
    return s, gf, bf


def weight_column_max(weights: Sequence[torch.Tensor], w_max=None, stream=None) -> torch.Tensor:
    """max over the weights and their rows of |W[n, j]|, per input column j."""
    K = weights[0].shape[1]
    dt = _dtype_code(weights[0])
    for w in weights:
        _rows(w, "W")
        if not w.is_contiguous() or w.shape[1] != K or _dtype_code(w) != dt:
            raise ValueError("weights must be contiguous [N, K] of one dtype")
    ptrs = (ctypes.c_void_p * len(weights))(*[w.data_ptr() for w in weights])
    ns = (ctypes.c_int64 * len(weights))(*[w.shape[0] for w in weights])
    with _scope(weights[0].device, stream):
        if w_max is None:
            w_max = torch.empty(K, dtype=torch.float32, device=weights[0].device)
        _check(lib().sq_weight_column_max(ctypes.cast(ptrs, ctypes.c_void_p),
                                          ctypes.cast(ns, ctypes.c_void_p), len(weights), dt, K,
                                          _ptr(_vec(w_max, K, "w_max")), _stream(stream)),
               "sq_weight_column_max")
    return w_max


def smooth_scales_from_maxima(act_max: torch.Tensor, w_max: torch.Tensor, alpha: float,
                              clamp_eps: float = 1e-5, gamma=None, beta=None, s=None,
                              gamma_folded=None, beta_folded=None, stream=None):
    """s, gamma / s and beta / s from the two maxima (s may be w_max)."""
    K = act_max.numel()
    dev = act_max.device
    with _scope(dev, stream):
        s = torch.empty(K, dtype=torch.float32, device=dev) if s is None else s
        gf = (torch.empty(K, dtype=torch.float32, device=dev) if gamma_folded is None
              else gamma_folded)
        bf = None
        if beta is not None:
            bf = (torch.empty(K, dtype=torch.float32, device=dev) if beta_folded is None
                  else beta_folded)
        _check(lib().sq_smooth_scales_from_maxima(
            _ptr(_vec(act_max, K, "act_max")), _ptr(_vec(w_max, K, "w_max")), K, float(alpha),
            clamp_eps, _ptr(_vec(gamma, K, "gamma")), _ptr(_vec(beta, K, "beta")),
            _ptr(_vec(s, K, "s")), _ptr(_vec(gf, K, "gamma_folded")),
            _ptr(_vec(bf, K, "beta_folded")), _stream(stream)), "sq_smooth_scales_from_maxima")
    return s, gf, bf


def smooth_quantize_weights(W: torch.Tensor, s: Optional[torch.Tensor] = None, Wq=None,
                            w_scale=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    N, K, ld = _rows(W, "W")
    with _scope(W.device, stream):
        if Wq is None:
            Wq = torch.empty((N, K), dtype=torch.int8, device=W.device)
        if w_scale is None:
            w_scale = torch.empty(N, dtype=torch.float32, device=W.device)
        _check(lib().sq_smooth_quantize_weights(_ptr(W), _dtype_code(W), N, K, ld,
                                                _ptr(_vec(s, K, "s")), _ptr(Wq), _ptr(w_scale),
                                                _stream(stream)), "sq_smooth_quantize_weights")
    return Wq, w_scale


def norm_smooth_quant_per_token(x: torch.Tensor, norm: int, gamma_folded=None, beta_folded=None,
                                eps: float = 1e-5, Xq=None, x_scale=None, stream=None
                                ) -> Tuple[torch.Tensor, torch.Tensor]:
    M, K, ld = _rows(x, "x")
    with _scope(x.device, stream):
        if Xq is None:
            Xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
        if x_scale is None:
            x_scale = torch.empty(M, dtype=torch.float32, device=x.device)
        _check(lib().sq_norm_smooth_quant_per_token(
            _ptr(x), _dtype_code(x), M, K, ld, norm, _ptr(_vec(gamma_folded, K, "gamma_folded")),
            _ptr(_vec(beta_folded, K, "beta_folded")), eps, _ptr(Xq), _ptr(x_scale),
            _stream(stream)), "sq_norm_smooth_quant_per_token")
    return Xq, x_scale


def norm_smooth_absmax(x: torch.Tensor, norm: int, gamma_folded=None, beta_folded=None,
                       eps: float = 1e-5, absmax=None, stream=None) -> torch.Tensor:
    """Running max over all of |norm(x)| into a 1-element fp32 device tensor."""
    M, K, ld = _rows(x, "x")
    with _scope(x.device, stream):
        if absmax is None:
            absmax = torch.zeros(1, dtype=torch.float32, device=x.device)
        _check(lib().sq_norm_smooth_absmax(_ptr(x), _dtype_code(x), M, K, ld, norm,
                                           _ptr(_vec(gamma_folded, K, "gamma_folded")),
                                           _ptr(_vec(beta_folded, K, "beta_folded")), eps,
                                           _ptr(absmax), _stream(stream)), "sq_norm_smooth_absmax")
    return absmax


def norm_smooth_quant_per_tensor(x: torch.Tensor, norm: int, absmax: torch.Tensor,
                                 gamma_folded=None, beta_folded=None, eps: float = 1e-5,
                                 Xq=None, x_scale=None, stream=None):
    """Codes with the one step fl32(absmax / 127); x_scale holds it per row."""
    M, K, ld = _rows(x, "x")
    with _scope(x.device, stream):
        if Xq is None:
            Xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
        if x_scale is None:
            x_scale = torch.empty(M, dtype=torch.float32, device=x.device)
        _check(lib().sq_norm_smooth_quant_per_tensor(
            _ptr(x), _dtype_code(x), M, K, ld, norm, _ptr(_vec(gamma_folded, K, "gamma_folded")),
            _ptr(_vec(beta_folded, K, "beta_folded")), eps, _ptr(absmax), _ptr(Xq), _ptr(x_scale),
            _stream(stream)), "sq_norm_smooth_quant_per_tensor")
    return Xq, x_scale


def quant_per_token_given_absmax(x: torch.Tensor, row_absmax: torch.Tensor, Xq=None,
                                 x_scale=None, stream=None):
    """Per-token codes of x [M, K] with each row's max |x| given (no norm)."""
    M, K, ld = _rows(x, "x")
    with _scope(x.device, stream):
        if Xq is None:
            Xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
        if x_scale is None:
            x_scale = torch.empty(M, dtype=torch.float32, device=x.device)
        _check(lib().sq_quant_per_token_given_absmax(
            _ptr(x), _dtype_code(x), M, K, ld, _ptr(_vec(row_absmax, M, "row_absmax")), _ptr(Xq),
            _ptr(x_scale), _stream(stream)), "sq_quant_per_token_given_absmax")
    return Xq, x_scale


def row_absmax(x: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """max_k |x[m, k]| per row of x [M, K] (no norm), fp32 [M]."""
    M, K, ld = _rows(x, "x")
    with _scope(x.device, stream):
        if out is None:
            out = torch.empty(M, dtype=torch.float32, device=x.device)
        _check(lib().sq_row_absmax(_ptr(x), _dtype_code(x), M, K, ld, _ptr(_vec(out, M, "out")),
                                   _stream(stream)), "sq_row_absmax")
    return out


def dequant_i32(acc: torch.Tensor, x_scale: torch.Tensor, w_scale: torch.Tensor,
                epi: str = "bf16", out=None, stream=None) -> torch.Tensor:
    """The GEMM's epilogue on an INT32 accumulator acc [M, N]: bf16 [M, N]."""
    if acc.dim() != 2 or acc.dtype != torch.int32 or (acc.shape[1] > 1 and acc.stride(1) != 1):
        raise ValueError("acc must be an int32 [M, N] tensor with unit column stride")
    M, N = acc.shape
    if epi not in ("bf16", "bf16_relu"):
        raise ValueError("epi must be bf16 or bf16_relu")
    with _scope(acc.device, stream):
        if out is None:
            out = torch.empty((M, N), dtype=torch.bfloat16, device=acc.device)
        if tuple(out.shape) != (M, N) or out.dtype != torch.bfloat16 or \
                (N > 1 and out.stride(1) != 1):
            raise ValueError("out must be a bf16 [M, N] tensor with unit column stride")
        _check(lib().sq_dequant_i32(_ptr(acc), M, N, max(acc.stride(0), N),
                                    _ptr(_vec(x_scale, M, "x_scale")),
                                    _ptr(_vec(w_scale, N, "w_scale")), EPI[epi], _ptr(out),
                                    max(out.stride(0), N), _stream(stream)), "sq_dequant_i32")
    return out


def llmint8_outliers(col_absmax: torch.Tensor, tau: float = 6.0, mask=None, idx=None, count=None,
                     stream=None):
    """(mask [K] fp32, idx [K] int32, count [1] int32) of the LLM.int8()
    comparator: mask 0 on the channels with col_absmax >= tau, idx[:count] those
    channels ascending (count stays on the device)."""
    K = col_absmax.numel()
    dev = col_absmax.device
    with _scope(dev, stream):
        if mask is None:
            mask = torch.empty(K, dtype=torch.float32, device=dev)
        if idx is None:
            idx = torch.empty(K, dtype=torch.int32, device=dev)
        if count is None:
            count = torch.empty(1, dtype=torch.int32, device=dev)
        if idx.dtype != torch.int32 or idx.numel() < K or count.dtype != torch.int32:
            raise ValueError("idx [K] and count [1] must be int32")
        _check(lib().sq_llmint8_outliers(_ptr(_vec(col_absmax, K, "col_absmax")), K, tau,
                                         _ptr(_vec(mask, K, "mask")), _ptr(idx), _ptr(count),
                                         _stream(stream)), "sq_llmint8_outliers")
    return mask, idx, count


def llmint8_combine(acc: torch.Tensor, x_scale, w_scale, x: torch.Tensor, W: torch.Tensor, idx,
                    count, epi: str = "bf16", out=None, stream=None) -> torch.Tensor:
    """The comparator's merge: the INT8 lane's epilogue plus the 16-bit lane
    over the outlier channels, bf16 [M, N]."""
    M, N = acc.shape
    _, K, ldx = _rows(x, "x")
    _, Kw, ldw = _rows(W, "W")
    if Kw != K or W.shape[0] != N or acc.dtype != torch.int32 or \
            (N > 1 and acc.stride(1) != 1):
        raise ValueError("acc [M, N] int32, x [M, K], W [N, K]")
    with _scope(acc.device, stream):
        if out is None:
            out = torch.empty((M, N), dtype=torch.bfloat16, device=acc.device)
        _check(lib().sq_llmint8_combine(_ptr(acc), M, N, max(acc.stride(0), N),
                                        _ptr(_vec(x_scale, M, "x_scale")),
                                        _ptr(_vec(w_scale, N, "w_scale")), _ptr(x), _dtype_code(x),
                                        ldx, _ptr(W), _dtype_code(W), ldw, K, _ptr(idx),
                                        _ptr(count), EPI[epi], _ptr(out), max(out.stride(0), N),
                                        _stream(stream)), "sq_llmint8_combine")
    return out


def silu_mul_quant_per_token(gate_up: torch.Tensor, Xq=None, x_scale=None, h_out=None,
                             stream=None, fp8: bool = False):
    """Per-token codes of h = SiLU(gate) * up from gate_up [M, 2I] (gate in the
    first I columns): INT8, or with ``fp8`` e4m3 bytes (uint8).  ``h_out``
    (bf16 [M, I]) also receives h when given."""
    M, K2, ld = _rows(gate_up, "gate_up")
    if K2 % 2:
        raise ValueError("gate_up rows hold two halves")
    I = K2 // 2
    with _scope(gate_up.device, stream):
        if Xq is None:
            Xq = torch.empty((M, I), dtype=torch.uint8 if fp8 else torch.int8,
                             device=gate_up.device)
        if x_scale is None:
            x_scale = torch.empty(M, dtype=torch.float32, device=gate_up.device)
        ldh = 0
        if h_out is not None:
            if h_out.dtype != torch.bfloat16 or tuple(h_out.shape) != (M, I):
                raise ValueError("h_out must be bf16 [M, I]")
            _, _, ldh = _rows(h_out, "h_out")
        call = "sq_silu_mul_quant_per_token_fp8" if fp8 else "sq_silu_mul_quant_per_token"
        _check(getattr(lib(), call)(_ptr(gate_up), _dtype_code(gate_up), M, I, ld, _ptr(Xq),
                                    _ptr(x_scale), _ptr(h_out), ldh, _stream(stream)), call)
    return Xq, x_scale


# ---- FP8 (e4m3) W8A8: codes are uint8 tensors holding e4m3 bytes ----------

def norm_smooth_quant_per_token_fp8(x: torch.Tensor, norm: int, gamma_folded=None,
                                    beta_folded=None, eps: float = 1e-5, Xq8=None, x_scale=None,
                                    stream=None):
    M, K, ld = _rows(x, "x")
    with _scope(x.device, stream):
        if Xq8 is None:
            Xq8 = torch.empty((M, K), dtype=torch.uint8, device=x.device)
        if x_scale is None:
            x_scale = torch.empty(M, dtype=torch.float32, device=x.device)
        _check(lib().sq_norm_smooth_quant_per_token_fp8(
            _ptr(x), _dtype_code(x), M, K, ld, norm, _ptr(_vec(gamma_folded, K, "gamma_folded")),
            _ptr(_vec(beta_folded, K, "beta_folded")), eps, _ptr(Xq8), _ptr(x_scale),
            _stream(stream)), "sq_norm_smooth_quant_per_token_fp8")
    return Xq8, x_scale


def smooth_quantize_weights_fp8(W: torch.Tensor, s: Optional[torch.Tensor] = None, Wq8=None,
                                w_scale=None, stream=None):
    N, K, ld = _rows(W, "W")
    with _scope(W.device, stream):
        if Wq8 is None:
            Wq8 = torch.empty((N, K), dtype=torch.uint8, device=W.device)
        if w_scale is None:
            w_scale = torch.empty(N, dtype=torch.float32, device=W.device)
        _check(lib().sq_smooth_quantize_weights_fp8(_ptr(W), _dtype_code(W), N, K, ld,
                                                    _ptr(_vec(s, K, "s")), _ptr(Wq8), _ptr(w_scale),
                                                    _stream(stream)),
               "sq_smooth_quantize_weights_fp8")
    return Wq8, w_scale


def fp8_gemm_dequant(Xq8: torch.Tensor, Wq8: torch.Tensor, x_scale: Optional[torch.Tensor],
                     w_scale: Optional[torch.Tensor], epi: str = "bf16", out=None,
                     path_hint: int = 0, workspace=None, whole_k: bool = False,
                     stream=None) -> torch.Tensor:
    """e4m3 GEMM with the dequant epilogue.  Decode tiles run stream-K with a
    workspace (allocated here when not given) unless ``whole_k``."""
    M, K = Xq8.shape
    N = Wq8.shape[0]
    if Xq8.dtype != torch.uint8 or Wq8.dtype != torch.uint8 or not Xq8.is_contiguous() \
            or not Wq8.is_contiguous() or Wq8.shape[1] != K:
        raise ValueError("Xq8 [M,K] and Wq8 [N,K] must be contiguous uint8 (e4m3 bytes)")
    with _scope(Xq8.device, stream):
        if out is None:
            out = torch.empty((M, N), dtype=torch.float32 if epi == "f32" else torch.bfloat16,
                              device=Xq8.device)
        if whole_k:
            workspace = None
        else:
            need = gemm_workspace_size(M, N, K, 0) if path_hint != 1 and path_hint != 3 else 0
            if workspace is None and need:
                workspace = torch.empty(need, dtype=torch.uint8, device=Xq8.device)
        wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
        _check(lib().sq_fp8_gemm_dequant(_ptr(Xq8), _ptr(Wq8), _ptr(x_scale), _ptr(w_scale), M, N,
                                         K, EPI[epi], _ptr(out), out.stride(0), _ptr(workspace), wsb,
                                         path_hint, _stream(stream)), "sq_fp8_gemm_dequant")
    return out


def smooth_quantize_weights_per_tensor(W: torch.Tensor, s: Optional[torch.Tensor] = None,
                                       Wq=None, w_scale=None, w_absmax=None, stream=None):
    N, K, ld = _rows(W, "W")
    with _scope(W.device, stream):
        if Wq is None:
            Wq = torch.empty((N, K), dtype=torch.int8, device=W.device)
        if w_scale is None:
            w_scale = torch.empty(N, dtype=torch.float32, device=W.device)
        if w_absmax is None:
            w_absmax = torch.empty(1, dtype=torch.float32, device=W.device)
        _check(lib().sq_smooth_quantize_weights_per_tensor(
            _ptr(W), _dtype_code(W), N, K, ld, _ptr(_vec(s, K, "s")), _ptr(Wq), _ptr(w_scale),
            _ptr(w_absmax), _stream(stream)), "sq_smooth_quantize_weights_per_tensor")
    return Wq, w_scale


def gemm_plan(M: int, N: int, K: int, path_hint: int = 0, split_k: int = 0) -> GemmPlanInfo:
    info = GemmPlanInfo()
    _check(lib().sq_w8a8_gemm_plan(M, N, K, path_hint, split_k, ctypes.byref(info)),
           "sq_w8a8_gemm_plan")
    return info


def gemm_workspace_size(M: int, N: int, K: int, split_k: int = 0) -> int:
    return int(lib().sq_w8a8_gemm_workspace_size(M, N, K, split_k))


def w8a8_gemm_dequant(Xq: torch.Tensor, Wq: torch.Tensor, x_scale: Optional[torch.Tensor],
                      w_scale: Optional[torch.Tensor], epi: str = "bf16", out=None,
                      path_hint: int = 0, split_k: int = 0, workspace=None, stream=None
                      ) -> torch.Tensor:
    M, K = Xq.shape
    N = Wq.shape[0]
    if Xq.dtype != torch.int8 or Wq.dtype != torch.int8 or not Xq.is_contiguous() \
            or not Wq.is_contiguous() or Wq.shape[1] != K:
        raise ValueError("Xq [M,K] and Wq [N,K] must be contiguous int8")
    code = EPI[epi]
    with _scope(Xq.device, stream):
        if out is None:
            out = torch.empty((M, N), dtype=torch.int32 if epi == "i32" else torch.bfloat16,
                              device=Xq.device)
        need = gemm_workspace_size(M, N, K, split_k)
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=Xq.device)
        wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
        _check(lib().sq_w8a8_gemm_dequant(_ptr(Xq), _ptr(Wq), _ptr(x_scale), _ptr(w_scale), M, N, K,
                                          code, _ptr(out), out.stride(0), _ptr(workspace), wsb,
                                          path_hint, split_k, _stream(stream)),
               "sq_w8a8_gemm_dequant")
    return out


def w8a8_gemm_dequant_rowmax(Xq: torch.Tensor, Wq: torch.Tensor, x_scale: torch.Tensor,
                             w_scale: torch.Tensor, epi: str = "bf16", out=None,
                             row_absmax=None, path_hint: int = 0, stream=None):
    """The prefill GEMM that also returns max_n |out[m, n]| per row (bf16
    epilogues only).  Returns (out, row_absmax)."""
    M, K = Xq.shape
    N = Wq.shape[0]
    if Xq.dtype != torch.int8 or Wq.dtype != torch.int8 or not Xq.is_contiguous() \
            or not Wq.is_contiguous() or Wq.shape[1] != K:
        raise ValueError("Xq [M,K] and Wq [N,K] must be contiguous int8")
    with _scope(Xq.device, stream):
        if out is None:
            out = torch.empty((M, N), dtype=torch.bfloat16, device=Xq.device)
        if row_absmax is None:
            row_absmax = torch.empty(M, dtype=torch.float32, device=Xq.device)
        _check(lib().sq_w8a8_gemm_dequant_rowmax(
            _ptr(Xq), _ptr(Wq), _ptr(x_scale), _ptr(w_scale), M, N, K, EPI[epi], _ptr(out),
            out.stride(0), _ptr(_vec(row_absmax, M, "row_absmax")), path_hint, _stream(stream)),
            "sq_w8a8_gemm_dequant_rowmax")
    return out, row_absmax


def w8a8_gemm_dequant_noalloc(Xq: torch.Tensor, Wq: torch.Tensor,
                              x_scale: Optional[torch.Tensor], w_scale: Optional[torch.Tensor],
                              out: torch.Tensor, epi: str = "bf16", path_hint: int = 0,
                              split_k: int = 0, stream=None) -> torch.Tensor:
    """The GEMM for callers that cannot allocate: the caller passes every input
    and the output; split-K scratch comes from the library's own fixed array
    (see include/sq.h).  Calls that overlap on the GPU share that array."""
    M, K = Xq.shape
    N = Wq.shape[0]
    if Xq.dtype != torch.int8 or Wq.dtype != torch.int8 or not Xq.is_contiguous() \
            or not Wq.is_contiguous() or Wq.shape[1] != K:
        raise ValueError("Xq [M,K] and Wq [N,K] must be contiguous int8")
    # the C ABI cannot see the output's extent: a wrong one would be written past
    want = torch.int32 if epi == "i32" else torch.bfloat16
    if (out.dim() != 2 or tuple(out.shape) != (M, N) or out.dtype != want
            or (N > 1 and out.stride(1) != 1) or out.stride(0) < N
            or out.device != Xq.device or Wq.device != Xq.device):
        raise ValueError("out must be a [M, N] = [%d, %d] %s tensor with unit column stride "
                         "on the device of Xq" % (M, N, want))
    with _scope(Xq.device, stream):
        _check(lib().sq_w8a8_gemm_dequant_noalloc(_ptr(Xq), _ptr(Wq), _ptr(x_scale), _ptr(w_scale),
                                                  M, N, K, EPI[epi], _ptr(out), out.stride(0),
                                                  path_hint, split_k, _stream(stream)),
               "sq_w8a8_gemm_dequant_noalloc")
    return out


def linear_w8a8(x: torch.Tensor, norm: int, gamma_folded, beta_folded, eps: float,
                Wq: torch.Tensor, w_scale: torch.Tensor, epi: str = "bf16", out=None,
                Xq_scratch=None, xscale_scratch=None, workspace=None, stream=None) -> torch.Tensor:
    M, K, ld = _rows(x, "x")
    N = Wq.shape[0]
    with _scope(x.device, stream):
        if out is None:
            out = torch.empty((M, N), dtype=torch.int32 if epi == "i32" else torch.bfloat16,
                              device=x.device)
        if Xq_scratch is None:
            Xq_scratch = torch.empty((M, K), dtype=torch.int8, device=x.device)
        if xscale_scratch is None:
            xscale_scratch = torch.empty(M, dtype=torch.float32, device=x.device)
        need = gemm_workspace_size(M, N, K, 0)
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
        _check(lib().sq_linear_w8a8(_ptr(x), _dtype_code(x), M, K, ld, norm,
                                    _ptr(_vec(gamma_folded, K, "gamma_folded")),
                                    _ptr(_vec(beta_folded, K, "beta_folded")), eps, _ptr(Wq),
                                    _ptr(w_scale), N, EPI[epi], _ptr(out), out.stride(0),
                                    _ptr(Xq_scratch), _ptr(xscale_scratch), _ptr(workspace), wsb,
                                    _stream(stream)), "sq_linear_w8a8")
    return out


# ---- layers of experts -----------------------------------------------------

class MoeRoute(NamedTuple):
    """What :func:`moe_route` gives: see sq_moe_route in include/sq.h."""
    weights: torch.Tensor    # [T, top_k] fp32
    experts: torch.Tensor    # [T, top_k] int32, -1: none
    offsets: torch.Tensor    # [E + 1] int32, expert e's rows are offsets[e] .. offsets[e + 1]
    row_token: torch.Tensor  # [T * top_k] int32, the token of each row
    token_row: torch.Tensor  # [T, top_k] int32, the row of each token's j-th expert, -1: none


def _dense(t: Optional[torch.Tensor], shape, dtype, device, name: str):
    """Address of a contiguous tensor of exactly this shape, type and device
    (None of None)."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s"
                         % (name, dtype, list(shape), device))
    return t.data_ptr()


def moe_route_workspace_size(T: int, E: int, top_k: int) -> int:
    return int(lib().sq_moe_route_workspace_size(T, E, top_k))


def moe_route(logits: torch.Tensor, top_k: int, score: str = "softmax", bias=None,
              renormalize: bool = True, scale: float = 1.0, weights=None, experts=None,
              offsets=None, row_token=None, token_row=None, workspace=None,
              stream=None) -> MoeRoute:
    """The top_k experts of every token from the router's logits [T, E] (fp32 or
    bf16), and the (token, expert) rows sorted by expert.  ``score``: "softmax"
    or "sigmoid"; ``bias`` [E] (sigmoid only) is added for the choice alone."""
    T, E, ld = _rows(logits, "logits")
    dev = logits.device
    if score not in MOE_SCORES:
        raise ValueError("score must be one of %s" % sorted(MOE_SCORES))
    if not 1 <= top_k <= E:
        raise ValueError("top_k must be 1 .. %d (the experts), got %d" % (E, top_k))
    f32, i32, empty, L = torch.float32, torch.int32, torch.empty, lib()
    bias_p = _dense(bias, (E,), f32, dev, "bias")
    _dense(weights, (T, top_k), f32, dev, "weights")
    _dense(experts, (T, top_k), i32, dev, "experts")
    _dense(offsets, (E + 1,), i32, dev, "offsets")
    _dense(row_token, (T * top_k,), i32, dev, "row_token")
    _dense(token_row, (T, top_k), i32, dev, "token_row")
    ws_p, wsb = None, 0
    with _scope(dev, stream):
        if weights is None:
            weights = empty(T, top_k, dtype=f32, device=dev)
        if experts is None:
            experts = empty(T, top_k, dtype=i32, device=dev)
        if offsets is None:
            offsets = empty(E + 1, dtype=i32, device=dev)
        if row_token is None:
            row_token = empty(T * top_k, dtype=i32, device=dev)
        if token_row is None:
            token_row = empty(T, top_k, dtype=i32, device=dev)
        if workspace is None:
            need = L.sq_moe_route_workspace_size(T, E, top_k)
            if need:
                workspace = empty(need, dtype=torch.uint8, device=dev)
        if workspace is not None:
            if workspace.device != dev or not workspace.is_contiguous():
                raise ValueError("workspace must be contiguous and on the device of logits")
            ws_p, wsb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        _check(L.sq_moe_route(logits.data_ptr(), _dtype_code(logits), T, E, ld, top_k,
                              MOE_SCORES[score], bias_p, int(renormalize), scale,
                              weights.data_ptr(), experts.data_ptr(), offsets.data_ptr(),
                              row_token.data_ptr(), token_row.data_ptr(), ws_p, wsb,
                              _raw_stream(dev.index)), "sq_moe_route")
    return MoeRoute(weights, experts, offsets, row_token, token_row)


def _gemm_grouped(call: str, code: torch.dtype, raw: str, Xq, Wq, x_scale, w_scale, offsets,
                  row_token, epi, out, path_hint, stream):
    dev = Xq.device
    if Xq.dim() != 2 or Wq.dim() != 3 or Wq.shape[2] != Xq.shape[1] or Xq.dtype != code \
            or Wq.dtype != code or not Xq.is_contiguous() or not Wq.is_contiguous() \
            or not Xq.is_cuda or Wq.device != dev:
        raise ValueError("Xq [X,K] and Wq [E,N,K] must be contiguous %s tensors on one CUDA "
                         "device" % code)
    X, K = Xq.shape
    E, N, _ = Wq.shape
    if epi not in ("bf16", "bf16_relu", raw):
        raise ValueError("epi must be bf16, bf16_relu or %s" % raw)
    want = torch.bfloat16 if epi != raw else torch.int32 if raw == "i32" else torch.float32
    R = X if row_token is None else row_token.numel()
    off_p = _dense(offsets, (E + 1,), torch.int32, dev, "offsets")
    row_p = _dense(row_token, (R,), torch.int32, dev, "row_token")
    xs_p = _dense(x_scale, (X,), torch.float32, dev, "x_scale")
    ws_p = _dense(w_scale, (E, N), torch.float32, dev, "w_scale")
    L = lib()
    with _scope(dev, stream):
        ldo = N
        if out is None:
            out = torch.empty(R, N, dtype=want, device=dev)
        elif (out.dim() != 2 or out.shape != (R, N) or out.dtype != want or out.device != dev
              or (N > 1 and out.stride(1) != 1) or (R > 1 and out.stride(0) < N)):
            raise ValueError("out must be a [R, N] = [%d, %d] %s tensor with unit column stride "
                             "on the device of Xq" % (R, N, want))
        elif R > 1:
            ldo = out.stride(0)
        _check(getattr(L, call)(Xq.data_ptr(), X, Wq.data_ptr(), xs_p, ws_p, off_p, row_p, R, E, N,
                                K, EPI[epi], out.data_ptr(), ldo, path_hint,
                                _raw_stream(dev.index)), call)
    return out


def w8a8_gemm_grouped(Xq: torch.Tensor, Wq: torch.Tensor, x_scale: Optional[torch.Tensor],
                      w_scale: Optional[torch.Tensor], offsets: torch.Tensor, row_token=None,
                      epi: str = "bf16", out=None, path_hint: int = 0, stream=None
                      ) -> torch.Tensor:
    """Rows grouped by expert times each expert's weights: out[r] = row
    ``row_token[r]`` (or r) of Xq [X, K] by Wq[e] ([E, N, K]) for offsets[e] <=
    r < offsets[e + 1], dequantised to bf16 ("i32": the accumulator).  Rows of
    ``out`` behind offsets[E] are left as they were."""
    return _gemm_grouped("sq_w8a8_gemm_grouped", torch.int8, "i32", Xq, Wq, x_scale, w_scale,
                         offsets, row_token, epi, out, path_hint, stream)


def fp8_gemm_grouped(Xq8: torch.Tensor, Wq8: torch.Tensor, x_scale: Optional[torch.Tensor],
                     w_scale: Optional[torch.Tensor], offsets: torch.Tensor, row_token=None,
                     epi: str = "bf16", out=None, path_hint: int = 0, stream=None
                     ) -> torch.Tensor:
    """:func:`w8a8_gemm_grouped` on e4m3 bytes (uint8); "f32": the accumulator."""
    return _gemm_grouped("sq_fp8_gemm_grouped", torch.uint8, "f32", Xq8, Wq8, x_scale, w_scale,
                         offsets, row_token, epi, out, path_hint, stream)


def block_norm_quant_per_token(x: torch.Tensor, residual: Optional[torch.Tensor] = None, *,
                               token_row=None, weights=None, post_norm: int = NORM_NONE,
                               post_gamma=None, post_beta=None, post_eps: float = 1e-5,
                               gate=None, token_gate=None, residual_scale: float = 1.0,
                               pre_norm: int = NORM_RMS, pre_gamma=None, pre_beta=None,
                               pre_eps: float = 1e-5, fp8: bool = False, quant: bool = True,
                               h_out=None, Xq=None, x_scale=None, stream=None):
    """(h, Xq, x_scale) of the end of one block and the start of the next:
    h = residual_scale * residual + post_norm(x) * gate * token_gate, codes of
    pre_norm(h) per token.  With ``token_row`` and ``weights`` [M, top_k] x holds
    the experts' rows [R, K] and each token's are summed first.  ``h_out`` may be
    ``residual`` itself; without ``quant`` only h is computed (None, None)."""
    R, K, ldx = _rows(x, "x")
    dev, dt, f32, empty = x.device, x.dtype, torch.float32, torch.empty
    M, top_k, row_p, w_p = R, 0, None, None
    if (token_row is None) != (weights is None):
        raise ValueError("token_row and weights go together")
    if token_row is not None:
        if token_row.dim() != 2:
            raise ValueError("token_row must be [M, top_k]")
        M, top_k = token_row.shape
        row_p = _dense(token_row, (M, top_k), torch.int32, dev, "token_row")
        w_p = _dense(weights, (M, top_k), f32, dev, "weights")
    vec = (K,)
    post_g = _dense(post_gamma, vec, f32, dev, "post_gamma")
    post_b = _dense(post_beta, vec, f32, dev, "post_beta")
    gate_p = _dense(gate, vec, f32, dev, "gate")
    token_p = _dense(token_gate, (M,), f32, dev, "token_gate")
    pre_g = _dense(pre_gamma, vec, f32, dev, "pre_gamma")
    pre_b = _dense(pre_beta, vec, f32, dev, "pre_beta")
    res_p, ld_res, ld_h = None, K, K
    for name, v in (("residual", residual), ("h_out", h_out)):
        if v is not None and (v.shape != (M, K) or v.dtype != dt or v.device != dev):
            raise ValueError("%s must be [%d, %d] %s on the device of x" % (name, M, K, dt))
    if residual is not None:
        res_p, ld_res = residual.data_ptr(), _rows(residual, "residual")[2]
    if h_out is not None:
        ld_h = _rows(h_out, "h_out")[2]
    code = torch.uint8 if fp8 else torch.int8
    _dense(Xq, (M, K), code, dev, "Xq")
    _dense(x_scale, (M,), f32, dev, "x_scale")
    call = "sq_block_norm_quant_per_token_fp8" if fp8 else "sq_block_norm_quant_per_token"
    L = lib()
    with _scope(dev, stream):
        if h_out is None:
            h_out = empty(M, K, dtype=dt, device=dev)
        q_p = s_p = None
        if quant:
            if Xq is None:
                Xq = empty(M, K, dtype=code, device=dev)
            if x_scale is None:
                x_scale = empty(M, dtype=f32, device=dev)
            q_p, s_p = Xq.data_ptr(), x_scale.data_ptr()
        else:
            Xq = x_scale = None
        if M == 0:
            return h_out, Xq, x_scale
        a = BlockNormArgs(x.data_ptr(), ldx, R, row_p, w_p, top_k, _dtype_code(x), M, K, post_norm,
                          post_g, post_b, post_eps, gate_p, token_p, res_p, ld_res,
                          residual_scale, pre_norm, pre_g, pre_b, pre_eps, h_out.data_ptr(), ld_h,
                          q_p, s_p)
        _check(getattr(L, call)(ctypes.byref(a), _raw_stream(dev.index)), call)
    return h_out, Xq, x_scale


def get_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error word."""
    return int(lib().sq_get_device_error(_stream(stream)))


def set_wait_limit(polls: int) -> None:
    lib().sq_set_wait_limit(int(polls))


def status_string(status: int) -> str:
    return _status_text(status)
