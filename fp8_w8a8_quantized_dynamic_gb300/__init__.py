"""FP8 (e4m3fn) W8A8 linear with dynamic per-tensor activation quantization, for sm_103a.

Thin ctypes binding over the C-ABI library libfp8w8a8.so (declared in include/fp8w8a8.h).
The functions carry the C names. PyTorch supplies device memory and the current CUDA
stream only; every step of the layer runs in the library's CUDA kernels. There is no CPU
fallback: a missing library raises.

Typical use::

    qw, s_w = fp8_quantize_weight(w)                 # once, at load (per-tensor)
    qw, s_w = fp8_quantize_weight(w, per_channel=True)
    y = fp8_linear(a, qw, s_w, bias)                 # every forward; dynamic s_a
    y = fp8_linear_channelwise(a, qw, s_w, bias)
    y = fp8_linear_static(a, s_a, qw, s_w)           # calibrated activation scale
    qw, s_w = fp8_quantize_weight(w, fmt="e5m2")     # the other FP8 format
    y = fp8_linear_ex(a, qw, s_w, fmt_a="e5m2", fmt_w="e5m2")
    y = fp8_linear_weight_only(a, qw, s_w, fmt_w="e5m2")  # bf16 A, FP8 weights up-converted
    qw, s_w = fp8_block_quantize_weight(w)           # a scale for each 128 x 128 block
    y = fp8_block_linear(a, qw, s_w, bias)           # activations: a scale per row and 128 columns
    ids, weights = fp8_moe_route(logits, k, score="sigmoid", renormalize=True)
    y = fp8_moe_experts(x, ids, weights, qw13, s13, qw2, s2)  # the chosen experts, block-scaled
    xs, pos, offsets = fp8_moe_dispatch(x, ids, E)   # or rows sorted by expert for other networks, and back
    y = fp8_moe_combine(ys, pos, weights)
    y = fp8_lora_add(y, x, a, b, request_adapters)   # adapters of many requests beside a projection
    qa, s_a, r = fp8_residual_norm_quantize(y, w_norm, residual=r)  # the next block's norm, quantized for it

Kernels are launched on the current CUDA device and its current stream; tensors of another device are refused
(ValueError).
"""

from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional, Tuple

from ._build import LIB_PATH

FP8_OK = 0
FP8_ERR_INVALID_ARG = 1
FP8_ERR_MISALIGNED = 2
FP8_ERR_WORKSPACE = 3
FP8_ERR_CUDA = 4
FP8_ERR_TIMEOUT = 5
FP8_ERR_UNSUPPORTED_DEVICE = 6
FP8_QUANT_WORKSPACE_BYTES = 4352
FP8_E4M3, FP8_E5M2 = 0, 1
_FORMATS = {"e4m3": FP8_E4M3, "e5m2": FP8_E5M2}
FP8_NOALLOC_SCRATCH_BYTES = 8 * 1024 * 1024

_lock = threading.Lock()
_lib: Optional[ctypes.CDLL] = None

_i64, _sz, _vp, _int = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int

_SIGNATURES = {
    "fp8_min_ld": (_i64, [_i64]),
    "fp8_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "fp8_uses_gemv": (_int, [_i64, _i64, _i64]),
    "fp8_set_gemv_max_m": (_int, [_int]),
    "fp8_quantize_weight": (_int, [_vp, _i64, _i64, _i64, _int, _vp, _i64, _vp, _vp, _sz, _vp]),
    "fp8_quantize_act": (_int, [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _sz, _vp]),
    "fp8_scaled_mm": (_int, [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _int, _vp, _vp, _i64, _vp]),
    "fp8_linear": (_int, [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _sz, _vp]),
    "fp8_linear_channelwise": (_int, [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _sz, _vp]),
    "fp8_linear_noalloc": (_int, [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _int, _vp, _vp, _i64, _vp]),
    "fp8_quantize_weight_ex": (_int, [_vp, _i64, _i64, _i64, _int, _int, _vp, _i64, _vp, _vp, _sz, _vp]),
    "fp8_quantize_act_ex": (_int, [_vp, _i64, _i64, _i64, _int, _vp, _vp, _i64, _vp, _vp, _sz, _vp]),
    "fp8_scaled_mm_ex": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _int, _i64, _i64, _vp, _int, _vp, _vp,
                                _i64, _vp]),
    "fp8_linear_static": (_int, [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _int, _vp, _vp, _i64, _vp,
                                 _sz, _vp]),
    "fp8_linear_ex": (_int, [_vp, _i64, _i64, _i64, _int, _vp, _vp, _int, _i64, _i64, _vp, _int, _vp, _vp, _i64,
                             _vp, _sz, _vp]),
    "fp8_weight_only_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "fp8_linear_weight_only": (_int, [_vp, _i64, _i64, _i64, _vp, _int, _i64, _i64, _vp, _int, _vp, _vp, _i64,
                                      _vp, _sz, _vp]),
    "fp8_gemm_config": (_int, [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _sz, _vp, _vp, _vp, _vp, _vp]),
    "fp8_gemm_plan_model": (_int, [_i64, _i64, _i64, _int, _int, _sz, _vp, _vp, _vp, _vp, _vp]),
    "fp8_gemv_plan_model": (_int, [_i64, _i64, _i64, _int, _int, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fp8_block_quantize_weight": (_int, [_vp, _i64, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp]),
    "fp8_block_quantize_act": (_int, [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp]),
    "fp8_block_scaled_mm": (_int, [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _i64, _vp]),
    "fp8_block_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "fp8_block_linear": (_int, [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _sz, _vp]),
    "fp8_moe_route": (_int, [_vp, _int, _i64, _i64, _i64, _int, _vp, _int, _int, _int, _int, ctypes.c_float, _vp,
                             _vp, _vp]),
    "fp8_moe_route_ex": (_int, [_vp, _int, _i64, _i64, _i64, _int, _vp, _int, _int, _int, _int, _int, ctypes.c_float,
                                _vp, _vp, _vp]),
    "fp8_moe_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64, _i64]),
    "fp8_moe_experts": (_int, [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _i64, _i64,
                               _vp, _i64, _vp, _sz, _vp]),
    "fp8_moe_dispatch_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "fp8_moe_dispatch": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _sz, _vp]),
    "fp8_moe_combine": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _i64, _vp]),
    "fp8_moe_combine_grad": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _vp]),
    "fp8_moe_dispatch_grad": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp]),
    "fp8_lora_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64, _i64]),
    "fp8_lora_add": (_int, [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _sz,
                            _vp]),
    "fp8_residual_norm": (_int, [_vp, _i64, _i64, _i64, _vp, _vp, _i64, ctypes.c_float, _vp, _i64, _vp, ctypes.c_float,
                                 _int, _vp, _i64, _vp, _i64, _vp]),
    "fp8_residual_norm_quantize": (_int, [_vp, _i64, _i64, _i64, _vp, _vp, _i64, ctypes.c_float, _vp, _i64, _vp,
                                          ctypes.c_float, _int, _vp, _i64, _vp, _i64, _vp, _i64, _vp]),
    "fp8_last_device_status": (_int, [_vp]),
    "fp8_selftest_timeout": (_int, [_i64, _vp]),
    "fp8_block_selftest_timeout": (_int, [_int, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _vp,
                                          _i64, _vp]),
    "fp8_lora_selftest_timeout": (_int, [_int, _vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp,
                                         _i64, _vp, _sz, _vp]),
    "fp8_status_string": (ctypes.c_char_p, [_int]),
}


class FP8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def lib() -> ctypes.CDLL:
    """The loaded C library; raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(f"FP8 CUDA library missing ({LIB_PATH}); build it with "
                                       "fp8_w8a8_quantized_dynamic_gb300._build.build()")
                L = ctypes.CDLL(LIB_PATH)
                for name, (res, args) in _SIGNATURES.items():
                    fn = getattr(L, name)
                    fn.restype = res
                    fn.argtypes = args
                _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().fp8_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != FP8_OK:
        raise FP8Error(status, where)


def min_ld(K: int) -> int:
    """Leading dimension (bytes) of the library's FP8 matrices: K rounded up to 16 (16 for K == 0)."""
    return (int(K) + 15) // 16 * 16 if K > 0 else 16


# ---------------------------------------------------------------------------
# torch-facing wrappers (torch is imported lazily: host-only users need none of it)
# ---------------------------------------------------------------------------

_torch_module = None
_raw_stream = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream_query(torch):
    """index -> the current stream of CUDA device `index`, which has to be the current device: kernels are
    launched there, and another device's stream would put them in no order with that device's work. The raw
    query takes a tenth of a microsecond where building a Stream object takes two, a good part of a small
    call's time."""
    stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

    def query(index):
        if index != current():
            raise ValueError(f"tensors are on cuda:{index} and the current device is cuda:{current()} "
                             f"(call within torch.cuda.device({index}))")
        return stream(index)
    return query


def _stream_ptr(t) -> int:
    global _raw_stream
    if _raw_stream is None:
        _raw_stream = _stream_query(_torch())
    return _raw_stream(t.get_device())


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check_bf16_2d(t, name: str):
    torch = _torch()
    if t.dtype != torch.bfloat16 or t.dim() != 2 or t.stride(1) != 1 or not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA bf16 matrix with unit column stride")


def _check_fp8_2d(t, K: int, name: str):
    torch = _torch()
    if t.dtype != torch.uint8 or t.dim() != 2 or t.stride(1) != 1 or not t.is_cuda or t.shape[1] < K:
        raise ValueError(f"{name}: expected a CUDA uint8 [rows, ld >= K] matrix")


def fp8_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().fp8_workspace_bytes(M, K, N))


def fp8_uses_gemv(M: int, K: int, N: int) -> bool:
    return bool(lib().fp8_uses_gemv(M, K, N))


def fp8_set_gemv_max_m(m: int) -> int:
    """Largest M that runs the decode GEMV (clamped to 0..16; m < 0 only queries); returns the previous value."""
    return int(lib().fp8_set_gemv_max_m(int(m)))


def fp8_min_ld(K: int) -> int:
    return int(lib().fp8_min_ld(K))


def fp8_status_string(status: int) -> str:
    return status_string(status)


def workspace(M: int, K: int, N: int, device):
    """Allocate a workspace big enough for fp8_linear on [M, K] x [N, K] (and any quantize call)."""
    torch = _torch()
    return torch.empty(fp8_workspace_bytes(M, K, N), dtype=torch.uint8, device=device)


def _fmt(name: str) -> int:
    if name not in _FORMATS:
        raise ValueError(f"unknown FP8 format {name!r} (expected 'e4m3' or 'e5m2')")
    return _FORMATS[name]


def fp8_quantize_weight(w, per_channel: bool = False, ws=None, fmt: str = "e4m3"
                        ) -> Tuple["torch.Tensor", "torch.Tensor"]:
    """W bf16 [N, K] -> (qW uint8 [N, min_ld(K)], s_w fp32 [1] or [N]); fmt 'e4m3' or 'e5m2'."""
    torch = _torch()
    _check_bf16_2d(w, "w")
    N, K = w.shape
    qw = torch.empty((N, min_ld(K)), dtype=torch.uint8, device=w.device)
    s_w = torch.empty((N if per_channel else 1,), dtype=torch.float32, device=w.device)
    if ws is None and not per_channel:
        ws = torch.empty(FP8_QUANT_WORKSPACE_BYTES, dtype=torch.uint8, device=w.device)
    args = (w.data_ptr(), N, K, w.stride(0), int(per_channel))
    tail = (qw.data_ptr(), qw.stride(0), s_w.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel(), _stream_ptr(w))
    if fmt == "e4m3":
        _check(lib().fp8_quantize_weight(*args, *tail), "fp8_quantize_weight")
    else:
        _check(lib().fp8_quantize_weight_ex(*args, _fmt(fmt), *tail), "fp8_quantize_weight_ex")
    return qw, s_w


def fp8_quantize_act(a, ws=None, fmt: str = "e4m3", s_static=None):
    """A bf16 [M, K] -> (qA uint8 [M, min_ld(K)], s_a fp32 [1]).

    Dynamic s_a = amax(A) / max(fmt), or the given static scale s_static (device fp32 [1]).
    """
    torch = _torch()
    _check_bf16_2d(a, "a")
    M, K = a.shape
    qa = torch.empty((M, min_ld(K)), dtype=torch.uint8, device=a.device)
    s_a = torch.empty((1,), dtype=torch.float32, device=a.device)
    if ws is None and s_static is None:
        ws = torch.empty(FP8_QUANT_WORKSPACE_BYTES, dtype=torch.uint8, device=a.device)
    if fmt == "e4m3" and s_static is None:
        _check(lib().fp8_quantize_act(a.data_ptr(), M, K, a.stride(0), qa.data_ptr(), qa.stride(0), s_a.data_ptr(),
                                      ws.data_ptr(), ws.numel(), _stream_ptr(a)), "fp8_quantize_act")
    else:
        _check(lib().fp8_quantize_act_ex(a.data_ptr(), M, K, a.stride(0), _fmt(fmt), _ptr(s_static), qa.data_ptr(),
                                         qa.stride(0), s_a.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel(),
                                         _stream_ptr(a)), "fp8_quantize_act_ex")
    return qa, s_a


def fp8_scaled_mm(qa, K: int, s_a, qw, s_w, per_channel: bool = False, bias=None, out=None,
                  fmt_a: str = "e4m3", fmt_w: str = "e4m3"):
    """Y = bf16(s_a * s_w * (qA @ qW^T) (+ bias)) on already-quantized operands."""
    torch = _torch()
    _check_fp8_2d(qa, K, "qa")
    _check_fp8_2d(qw, K, "qw")
    M, N = qa.shape[0], qw.shape[0]
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=qa.device)
    if fmt_a == "e4m3" and fmt_w == "e4m3":
        _check(lib().fp8_scaled_mm(qa.data_ptr(), M, K, qa.stride(0), s_a.data_ptr(), qw.data_ptr(), N,
                                   qw.stride(0), s_w.data_ptr(), int(per_channel), _ptr(bias), y.data_ptr(),
                                   y.stride(0), _stream_ptr(qa)), "fp8_scaled_mm")
    else:
        _check(lib().fp8_scaled_mm_ex(qa.data_ptr(), _fmt(fmt_a), M, K, qa.stride(0), s_a.data_ptr(), qw.data_ptr(),
                                      _fmt(fmt_w), N, qw.stride(0), s_w.data_ptr(), int(per_channel), _ptr(bias),
                                      y.data_ptr(), y.stride(0), _stream_ptr(qa)), "fp8_scaled_mm_ex")
    return y


def _linear(fn_name: str, a, qw, s_w, bias, out, ws):
    torch = _torch()
    _check_bf16_2d(a, "a")
    M, K = a.shape
    _check_fp8_2d(qw, K, "qw")
    N = qw.shape[0]
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    L = lib()
    if ws is None:
        need = L.fp8_workspace_bytes(M, K, N)
        ws = workspace(M, K, N, a.device) if need else None
    fn = getattr(L, fn_name)
    _check(fn(a.data_ptr(), M, K, a.stride(0), qw.data_ptr(), N, qw.stride(0), s_w.data_ptr(), _ptr(bias),
              y.data_ptr(), y.stride(0), _ptr(ws), 0 if ws is None else ws.numel(), _stream_ptr(a)), fn_name)
    return y


def fp8_linear(a, qw, s_w, bias=None, out=None, ws=None):
    """Dynamic W8A8 linear, per-tensor weight scale s_w [1]: Y = A W^T (+ bias), bf16 out."""
    return _linear("fp8_linear", a, qw, s_w, bias, out, ws)


def fp8_linear_channelwise(a, qw, s_w, bias=None, out=None, ws=None):
    """Dynamic W8A8 linear, per-output-channel weight scales s_w [N]."""
    return _linear("fp8_linear_channelwise", a, qw, s_w, bias, out, ws)


def fp8_quantize_weight_ex(w, fmt: str, per_channel: bool = False, ws=None):
    """fp8_quantize_weight with an explicit FP8 format."""
    return fp8_quantize_weight(w, per_channel=per_channel, ws=ws, fmt=fmt)


def fp8_quantize_act_ex(a, fmt: str, s_static=None, ws=None):
    """fp8_quantize_act with an explicit FP8 format and an optional static scale."""
    return fp8_quantize_act(a, ws=ws, fmt=fmt, s_static=s_static)


def fp8_scaled_mm_ex(qa, fmt_a: str, K: int, s_a, qw, fmt_w: str, s_w, per_channel: bool = False, bias=None,
                     out=None):
    """fp8_scaled_mm with the FP8 formats of both operands."""
    return fp8_scaled_mm(qa, K, s_a, qw, s_w, per_channel=per_channel, bias=bias, out=out, fmt_a=fmt_a,
                         fmt_w=fmt_w)


def _prologue(a, qw, out, ws):
    torch = _torch()
    _check_bf16_2d(a, "a")
    M, K = a.shape
    _check_fp8_2d(qw, K, "qw")
    N = qw.shape[0]
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    if ws is None:
        need = lib().fp8_workspace_bytes(M, K, N)
        ws = workspace(M, K, N, a.device) if need else None
    return M, K, N, y, ws


def fp8_linear_static(a, s_a, qw, s_w, per_channel: bool = False, bias=None, out=None, ws=None):
    """W8A8 linear with a static (calibrated) activation scale s_a (device fp32 [1])."""
    M, K, N, y, ws = _prologue(a, qw, out, ws)
    _check(lib().fp8_linear_static(a.data_ptr(), M, K, a.stride(0), s_a.data_ptr(), qw.data_ptr(), N, qw.stride(0),
                                   s_w.data_ptr(), int(per_channel), _ptr(bias), y.data_ptr(), y.stride(0),
                                   _ptr(ws), 0 if ws is None else ws.numel(), _stream_ptr(a)), "fp8_linear_static")
    return y


def fp8_linear_ex(a, qw, s_w, per_channel: bool = False, bias=None, out=None, ws=None,
                  fmt_a: str = "e4m3", fmt_w: str = "e4m3", s_static=None):
    """The general linear: FP8 formats of A and W, dynamic (s_static None) or static activation scale."""
    M, K, N, y, ws = _prologue(a, qw, out, ws)
    _check(lib().fp8_linear_ex(a.data_ptr(), M, K, a.stride(0), _fmt(fmt_a), _ptr(s_static), qw.data_ptr(),
                               _fmt(fmt_w), N, qw.stride(0), s_w.data_ptr(), int(per_channel), _ptr(bias),
                               y.data_ptr(), y.stride(0), _ptr(ws), 0 if ws is None else ws.numel(),
                               _stream_ptr(a)), "fp8_linear_ex")
    return y


def fp8_weight_only_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().fp8_weight_only_workspace_bytes(M, K, N))


def fp8_linear_weight_only(a, qw, s_w, per_channel: bool = False, bias=None, out=None, ws=None,
                           fmt_w: str = "e4m3"):
    """Weight-only FP8 linear: bf16 A times the exactly up-converted FP8 weights, scaled by s_w."""
    torch = _torch()
    _check_bf16_2d(a, "a")
    M, K = a.shape
    _check_fp8_2d(qw, K, "qw")
    N = qw.shape[0]
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    if ws is None:
        need = fp8_weight_only_workspace_bytes(M, K, N)
        ws = torch.empty(need, dtype=torch.uint8, device=a.device) if need else None
    _check(lib().fp8_linear_weight_only(a.data_ptr(), M, K, a.stride(0), qw.data_ptr(), _fmt(fmt_w), N,
                                        qw.stride(0), s_w.data_ptr(), int(per_channel), _ptr(bias), y.data_ptr(),
                                        y.stride(0), _ptr(ws), 0 if ws is None else ws.numel(), _stream_ptr(a)),
           "fp8_linear_weight_only")
    return y


def fp8_linear_noalloc(a, qw, s_w, per_channel: bool = False, bias=None, out=None):
    """The linear without a workspace, for callers that cannot allocate device memory.

    Uses the library's fixed scratch array (FP8_NOALLOC_SCRATCH_BYTES per GPU) instead of
    a caller workspace; calls that overlap on the GPU share it and race. Only `out` (when
    omitted) is allocated here, by torch, for convenience; pass `out` to allocate nothing.
    """
    torch = _torch()
    _check_bf16_2d(a, "a")
    M, K = a.shape
    _check_fp8_2d(qw, K, "qw")
    N = qw.shape[0]
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    _check(lib().fp8_linear_noalloc(a.data_ptr(), M, K, a.stride(0), qw.data_ptr(), N, qw.stride(0),
                                    s_w.data_ptr(), int(per_channel), _ptr(bias), y.data_ptr(), y.stride(0),
                                    _stream_ptr(a)), "fp8_linear_noalloc")
    return y


# ---------------------------------------------------------------------------
# block-scaled linear and mixture of experts
# ---------------------------------------------------------------------------

def _blocks(n: int) -> int:
    return (n + 127) // 128


def _row_stride(t, rows: int, width: int) -> int:
    """Leading dimension handed to C: the true stride between rows, so that C refuses rows that overlap
    (broadcast ones have stride 0). A single row's stride means nothing: the width stands for it."""
    return t.stride(-2) if rows > 1 else width or 1


def _out_bf16(out, M: int, N: int, like):
    if out is None:
        return _torch().empty((M, N), dtype=like.dtype, device=like.device)  # `like` is bf16
    _check_bf16_2d(out, "out")
    if out.shape != (M, N) or out.device != like.device:
        raise ValueError(f"out: expected [{M}, {N}] on {like.device}")
    return out


def _check_dense(t, dtype, shape, index: int, name: str):
    """A gap-free tensor of this dtype and shape on CUDA device `index`."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}")


def _check_rows(t, dtype, rows: int, cols: int, index: int, name: str):
    """A matrix of this dtype and shape with unit column stride on CUDA device `index`."""
    if t.dtype != dtype or t.shape != (rows, cols) or (cols > 1 and t.stride(1) != 1) or t.get_device() != index:
        raise ValueError(f"{name}: expected a {dtype} matrix [{rows}, {cols}] with unit column stride on cuda:{index}")


def _check_block_weight(qw, s_w, lead: tuple, N: int, K: int, index: int, name: str) -> int:
    """Codes [*lead, N, ld] and scales [*lead, blocks of N, blocks of K] as fp8_block_quantize_weight returns
    them; returns ld."""
    torch = _torch()
    ld = qw.shape[-1]
    if ld < K or ld % 16 or ld == 0:
        raise ValueError(f"{name}: expected uint8 codes [..., N, ld] with ld a multiple of 16 and at least {K}")
    _check_dense(qw, torch.uint8, (*lead, N, ld), index, name)
    _check_dense(s_w, torch.float32, (*lead, (N + 127) // 128, (K + 127) // 128), index, name + " scales")
    return ld


def _scratch(ws, need: int, like):
    """(address, bytes, tensor) of the caller's workspace, or of a fresh one (none where none is needed)."""
    torch = _torch()
    if ws is None:
        if not need:
            return None, 0, None
        ws = torch.empty(need, dtype=torch.uint8, device=like.device)
        return ws.data_ptr(), need, ws
    if ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.device != like.device:
        raise ValueError(f"ws: expected a contiguous uint8 tensor on {like.device}")
    return ws.data_ptr(), ws.numel(), ws


def fp8_block_quantize_weight(w):
    """W bf16 [..., N, K] -> (qW uint8 [..., N, min_ld(K)], s_w fp32 [..., ceil(N/128), ceil(K/128)]):
    one scale for each 128 x 128 block. Leading dimensions are separate matrices (experts)."""
    torch = _torch()
    if w.dtype != torch.bfloat16 or w.dim() < 2 or not w.is_cuda or w.stride(-1) != 1:
        raise ValueError("w: expected CUDA bf16 matrices [..., N, K] with unit column stride")
    lead, (N, K) = tuple(w.shape[:-2]), w.shape[-2:]
    if w.dim() > 3:
        w = w.reshape(-1, N, K)
    B = w.shape[0] if w.dim() == 3 else 1
    qw = torch.empty((*lead, N, min_ld(K)), dtype=torch.uint8, device=w.device)
    s_w = torch.empty((*lead, _blocks(N), _blocks(K)), dtype=torch.float32, device=w.device)
    _check(lib().fp8_block_quantize_weight(w.data_ptr(), B, N, K, _row_stride(w, N, K),
                                           w.stride(0) if w.dim() == 3 else 0, qw.data_ptr(), min_ld(K),
                                           s_w.data_ptr(), _stream_ptr(w)), "fp8_block_quantize_weight")
    return qw, s_w


def fp8_block_quantize_act(a):
    """A bf16 [M, K] -> (qA uint8 [M, min_ld(K)], s_a fp32 [ceil(K/128), M]): one scale per row and 128 columns.
    The rows of s_a start on 16-byte boundaries (the product copies them in whole pieces)."""
    torch = _torch()
    _check_bf16_2d(a, "a")
    M, K = a.shape
    qa = torch.empty((M, min_ld(K)), dtype=torch.uint8, device=a.device)
    s_a = torch.empty((_blocks(K), (M + 3) // 4 * 4), dtype=torch.float32, device=a.device)[:, :M]
    _check(lib().fp8_block_quantize_act(a.data_ptr(), M, K, _row_stride(a, M, K), qa.data_ptr(), qa.stride(0),
                                        s_a.data_ptr(), max(s_a.stride(0), 1), _stream_ptr(a)),
           "fp8_block_quantize_act")
    return qa, s_a


def fp8_block_scaled_mm(qa, K: int, s_a, qw, s_w, bias=None, out=None):
    """The block-scaled product on already-quantized operands (fp8_block_quantize_act / _weight), bf16 out."""
    torch = _torch()
    _check_fp8_2d(qa, K, "qa")
    M, N, index = qa.shape[0], qw.shape[-2], qa.get_device()
    if s_a.dtype != torch.float32 or s_a.shape != (_blocks(K), M) or s_a.get_device() != index or (
            s_a.numel() and s_a.stride(1) != 1):
        raise ValueError(f"s_a: expected fp32 [{_blocks(K)}, {M}] with unit column stride")
    ld = _check_block_weight(qw, s_w, (), N, K, index, "qw")
    if bias is not None:
        _check_dense(bias, torch.bfloat16, (N,), index, "bias")
    y = torch.empty((M, N), dtype=torch.bfloat16, device=qa.device) if out is None else _out_bf16(out, M, N, qa)
    _check(lib().fp8_block_scaled_mm(qa.data_ptr(), M, K, qa.stride(0), s_a.data_ptr(),
                                     _row_stride(s_a, s_a.shape[0], M), qw.data_ptr(), N, ld, s_w.data_ptr(),
                                     _ptr(bias), y.data_ptr(), _row_stride(y, M, N), _stream_ptr(qa)),
           "fp8_block_scaled_mm")
    return y


def fp8_block_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().fp8_block_workspace_bytes(M, K, N))


def fp8_block_linear(a, qw, s_w, bias=None, out=None, ws=None):
    """Block-scaled W8A8 linear, Y = A W^T (+ bias) in bf16: A is quantized with a scale per row and 128 columns,
    qw, s_w come from fp8_block_quantize_weight."""
    # a decode step's calls are as short as the checks around them: each tensor is asked once
    torch = _torch_module or _torch()
    if a.dtype is not torch.bfloat16 or a.dim() != 2 or not a.is_cuda:
        raise ValueError("a: expected a CUDA bf16 matrix with unit column stride")
    M, K = a.shape
    lda, unit = a.stride()
    if unit != 1:
        raise ValueError("a: expected a CUDA bf16 matrix with unit column stride")
    index = a.get_device()
    N = qw.shape[-2]
    ld = _check_block_weight(qw, s_w, (), N, K, index, "qw")
    if bias is not None:
        _check_dense(bias, torch.bfloat16, (N,), index, "bias")
    L = _lib or lib()
    need = L.fp8_block_workspace_bytes(M, K, N)
    wp, wn, ws = _scratch(ws, need, a) if need or ws is not None else (None, 0, None)
    if out is None:
        y, ldy = torch.empty((M, N), dtype=torch.bfloat16, device=a.device), N or 1
    else:
        y = _out_bf16(out, M, N, a)
        ldy = _row_stride(y, M, N)
    status = L.fp8_block_linear(a.data_ptr(), M, K, lda if M > 1 else K or 1, qw.data_ptr(), N, ld, s_w.data_ptr(),
                                None if bias is None else bias.data_ptr(), y.data_ptr(), ldy, wp, wn, _stream_ptr(a))
    if status:
        raise FP8Error(status, "fp8_block_linear")
    return y


_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"auto": 0, "max": 1}


def fp8_moe_route(logits, k: int, score: str = "softmax", bias=None, groups: int = 1,
                  keep_groups: Optional[int] = None, renormalize: bool = False, factor: float = 1.0,
                  group_score: str = "auto"):
    """Logits [T, E] (fp32 or bf16) -> (ids int32 [T, k], weights fp32 [T, k]): the k chosen experts of each
    token in descending order and their routing weights. score 'softmax' or 'sigmoid'; bias fp32 [E] steers the
    choice only; only the keep_groups best of `groups` groups of experts take part (default: all).
    group_score 'auto': a group's score is the sum of its two best choices (softmax without bias: its best one);
    'max': its best choice in every case, as published gates without a bias have it, for sigmoid too."""
    torch = _torch_module or _torch()
    bf16 = logits.dtype is torch.bfloat16
    if not (bf16 or logits.dtype is torch.float32) or logits.dim() != 2 or not logits.is_cuda:
        raise ValueError("logits: expected a CUDA fp32 or bf16 matrix with unit column stride")
    T, E = logits.shape
    ld, unit = logits.stride()
    if unit != 1 and E > 1:
        raise ValueError("logits: expected a CUDA fp32 or bf16 matrix with unit column stride")
    kind = _SCORES.get(score)
    if kind is None:
        raise ValueError(f"unknown score {score!r} (expected 'softmax' or 'sigmoid')")
    group_max = _GROUP_SCORES.get(group_score)
    if group_max is None:
        raise ValueError(f"unknown group_score {group_score!r} (expected 'auto' or 'max')")
    if bias is not None:
        _check_dense(bias, torch.float32, (E,), logits.get_device(), "bias")
    if k < 1:
        raise ValueError(f"k: expected at least 1, got {k}")
    device = logits.device
    ids = torch.empty((T, k), dtype=torch.int32, device=device)
    weights = torch.empty((T, k), dtype=torch.float32, device=device)
    L = _lib or lib()
    keep = groups if keep_groups is None else keep_groups
    bias_ptr = None if bias is None else bias.data_ptr()
    if group_max:
        status = L.fp8_moe_route_ex(logits.data_ptr(), bf16, T, E, ld if T > 1 else E, kind, bias_ptr, groups, keep, 1, k,
                                    1 if renormalize else 0, factor, ids.data_ptr(), weights.data_ptr(),
                                    _stream_ptr(logits))
    else:
        status = L.fp8_moe_route(logits.data_ptr(), bf16, T, E, ld if T > 1 else E, kind, bias_ptr, groups, keep, k,
                                 1 if renormalize else 0, factor, ids.data_ptr(), weights.data_ptr(),
                                 _stream_ptr(logits))
    if status:
        raise FP8Error(status, "fp8_moe_route")
    return ids, weights


def fp8_moe_route_ex(logits, k: int, group_score: str, score: str = "softmax", bias=None, groups: int = 1,
                     keep_groups: Optional[int] = None, renormalize: bool = False, factor: float = 1.0):
    """fp8_moe_route with an explicit rule of a group's score."""
    return fp8_moe_route(logits, k, score, bias, groups, keep_groups, renormalize, factor, group_score)


def fp8_moe_workspace_bytes(T: int, k: int, E: int, H: int, I: int) -> int:
    return int(lib().fp8_moe_workspace_bytes(T, k, E, H, I))


def fp8_moe_experts(x, ids, weights, qw13, s13, qw2, s2, out=None, ws=None):
    """The routed experts' gated networks, summed by routing weight, bf16 [T, H].

    x bf16 [T, H]; ids int32 and weights fp32 [T, k] (fp8_moe_route; ids outside [0, E) contribute nothing);
    qw13, s13 from fp8_block_quantize_weight of [E, 2, I, H] (gate, up), qw2, s2 of [E, H, I]."""
    torch = _torch_module or _torch()
    _check_bf16_2d(x, "x")
    T, H = x.shape
    if ids.dim() != 2 or qw13.dim() != 4:
        raise ValueError("expected ids [T, k] and qw13 [E, 2, I, ld]")
    E, _, I, _ = qw13.shape
    k, index = ids.shape[1], x.get_device()
    _check_dense(ids, torch.int32, (T, k), index, "ids")
    _check_dense(weights, torch.float32, (T, k), index, "weights")
    ld13 = _check_block_weight(qw13, s13, (E, 2), I, H, index, "qw13")
    ld2 = _check_block_weight(qw2, s2, (E,), H, I, index, "qw2")
    L = _lib or lib()
    wp, wn, ws = _scratch(ws, L.fp8_moe_workspace_bytes(T, k, E, H, I), x)
    y = _out_bf16(out, T, H, x)
    status = L.fp8_moe_experts(x.data_ptr(), T, H, _row_stride(x, T, H), ids.data_ptr(), weights.data_ptr(), k,
                               qw13.data_ptr(), ld13, s13.data_ptr(), qw2.data_ptr(), ld2, s2.data_ptr(), E, I,
                               y.data_ptr(), _row_stride(y, T, H), wp, wn, _stream_ptr(x))
    if status:
        raise FP8Error(status, "fp8_moe_experts")
    return y


# ---------------------------------------------------------------------------
# adapters beside a projection
# ---------------------------------------------------------------------------

def fp8_lora_workspace_bytes(M: int, K: int, N: int, L: int, r: int) -> int:
    return int(lib().fp8_lora_workspace_bytes(M, K, N, L, r))


def fp8_lora_add(y, x, a, b, ids, scales=None, out=None, ws=None):
    """The low-rank adapters of many requests beside a projection they share: y[m] + scales[e] * B[e] (A[e] x[m]) with
    e = ids[m], bf16 [M, N]. y [M, N] is the projection's output of x [M, K] (both bf16), a bf16 [L, r, K],
    b bf16 [L, N, r], ids int32 [M] (outside [0, L): no adapter, the row is y's), scales fp32 [L] or None (ones). out may
    be y."""
    torch = _torch_module or _torch()
    bf16 = torch.bfloat16
    if y.dtype is not bf16 or x.dtype is not bf16 or y.dim() != 2 or x.dim() != 2 or not y.is_cuda:
        raise ValueError("y, x: expected CUDA bf16 matrices with unit column stride")
    M, N = y.shape
    K = x.shape[1]
    ldy, unit_y = y.stride()
    ldx, unit_x = x.stride()
    if (unit_y != 1 and N > 1) or (unit_x != 1 and K > 1):
        raise ValueError("y, x: expected CUDA bf16 matrices with unit column stride")
    index = y.get_device()
    if x.shape[0] != M or x.get_device() != index:
        raise ValueError(f"x: expected [{M}, K] on cuda:{index}")
    if a.dim() != 3:
        raise ValueError("a: expected bf16 [L, r, K]")
    L, r, _ = a.shape
    _check_dense(a, bf16, (L, r, K), index, "a")
    _check_dense(b, bf16, (L, N, r), index, "b")
    _check_dense(ids, torch.int32, (M,), index, "ids")
    if scales is not None:
        _check_dense(scales, torch.float32, (L,), index, "scales")
    lb = _lib or lib()
    need = lb.fp8_lora_workspace_bytes(M, K, N, L, r)
    wp, wn, ws = _scratch(ws, need, y) if need or ws is not None else (None, 0, None)
    if out is None:
        o, ldo = torch.empty((M, N), dtype=bf16, device=y.device), N or 1
    else:
        o = _out_bf16(out, M, N, y)
        ldo = _row_stride(o, M, N)
    status = lb.fp8_lora_add(y.data_ptr(), M, N, ldy if M > 1 else N or 1, x.data_ptr(), K, ldx if M > 1 else K or 1,
                             a.data_ptr(), b.data_ptr(), L, r, ids.data_ptr(), None if scales is None else scales.data_ptr(),
                             o.data_ptr(), ldo, wp, wn, _stream_ptr(y))
    if status:
        raise FP8Error(status, "fp8_lora_add")
    return o


# ---------------------------------------------------------------------------
# tokens sorted by expert and back
# ---------------------------------------------------------------------------

def _check_rows_in(t, name: str):
    """A CUDA matrix of bf16 or fp32 with unit column stride; (1 for fp32, rows, columns, row stride)."""
    torch = _torch_module or _torch()
    f32 = t.dtype is torch.float32
    if not (f32 or t.dtype is torch.bfloat16) or t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA bf16 or fp32 matrix with unit column stride")
    rows, cols = t.shape
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name}: expected a CUDA bf16 or fp32 matrix with unit column stride")
    return 1 if f32 else 0, rows, cols, ld if rows > 1 else cols or 1


def _rows_out(out, rows: int, cols: int, like, name: str = "out"):
    """(tensor, row stride) of an output of `like`'s type."""
    if out is None:
        return (_torch_module or _torch()).empty((rows, cols), dtype=like.dtype, device=like.device), cols or 1
    _check_rows(out, like.dtype, rows, cols, like.get_device(), name)
    return out, _row_stride(out, rows, cols)


def _check_pairs(pos, weights, index: int):
    """(T, k) of pos int32 [T, k] and weights fp32 of the same shape, or None."""
    torch = _torch_module or _torch()
    if pos.dim() != 2:
        raise ValueError("pos: expected an int32 matrix [T, k]")
    shape = pos.shape
    _check_dense(pos, torch.int32, shape, index, "pos")
    if weights is not None:
        _check_dense(weights, torch.float32, shape, index, "weights")
    return shape


def fp8_moe_dispatch_workspace_bytes(T: int, k: int, E: int) -> int:
    return int(lib().fp8_moe_dispatch_workspace_bytes(T, k, E))


def fp8_moe_dispatch(x, ids, E: int, out=None, ws=None):
    """Tokens copied to rows sorted by expert: x [T, H] (bf16 or fp32), ids int32 [T, k] -> (xs [T * k, H],
    pos int32 [T, k], offsets int32 [E + 1]). xs[pos[t, j]] = x[t]; rows offsets[e] to offsets[e + 1] are expert e's, in
    the tokens' order. Ids outside [0, E) have pos -1 and no row; rows from offsets[E] on are not written."""
    torch = _torch_module or _torch()
    f32, T, H, ldx = _check_rows_in(x, "x")
    if ids.dim() != 2:
        raise ValueError("ids: expected an int32 matrix [T, k]")
    k = ids.shape[1]
    _check_dense(ids, torch.int32, (T, k), x.get_device(), "ids")
    if E < 1:
        raise ValueError(f"E: expected at least 1, got {E}")
    L = _lib or lib()
    need = L.fp8_moe_dispatch_workspace_bytes(T, k, E)
    wp, wn, ws = _scratch(ws, need, x) if need or ws is not None else (None, 0, None)
    xs, ldxs = _rows_out(out, T * k, H, x)
    pos = torch.empty((T, k), dtype=torch.int32, device=x.device)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=x.device)
    status = L.fp8_moe_dispatch(x.data_ptr(), f32, T, H, ldx, ids.data_ptr(), k, E, xs.data_ptr(), ldxs, pos.data_ptr(),
                                offsets.data_ptr(), wp, wn, _stream_ptr(x))
    if status:
        raise FP8Error(status, "fp8_moe_dispatch")
    return xs, pos, offsets


def fp8_moe_combine(ys, pos, weights=None, out=None):
    """The experts' rows back at their tokens: y[t] = sum_j weights[t, j] ys[pos[t, j]] in fp32 (weights None: ones),
    of ys' type (bf16 or fp32). Pairs with pos outside ys' rows contribute nothing."""
    f32, R, H, ldys = _check_rows_in(ys, "ys")
    T, k = _check_pairs(pos, weights, ys.get_device())
    y, ldy = _rows_out(out, T, H, ys)
    status = (_lib or lib()).fp8_moe_combine(ys.data_ptr(), f32, R, H, ldys, pos.data_ptr(), _ptr(weights), T, k,
                                             y.data_ptr(), ldy, _stream_ptr(ys))
    if status:
        raise FP8Error(status, "fp8_moe_combine")
    return y


def fp8_moe_combine_grad(dy, ys, pos, weights, out=None):
    """The gradient of fp8_moe_combine: (dys [R, H] with dys[pos[t, j]] = weights[t, j] dy[t], dw fp32 [T, k] with
    <dy[t], ys[pos[t, j]]>). No two pairs may have the same row (those of fp8_moe_dispatch do not). Rows of dys that no
    pair has are zeros; in a given out, which may be ys, they are not written."""
    torch = _torch_module or _torch()
    f32, T, H, lddy = _check_rows_in(dy, "dy")
    index = dy.get_device()
    _, R, _, ldys = _check_rows_in(ys, "ys")
    _check_rows(ys, dy.dtype, R, H, index, "ys")
    if weights is None or _check_pairs(pos, weights, index)[0] != T:
        raise ValueError("expected pos [T, k] and weights [T, k] for dy [T, H]")
    k = pos.shape[1]
    if out is None:  # (the kernel passes rows with a pair only)
        dys, lddys = torch.zeros((R, H), dtype=ys.dtype, device=ys.device), H or 1
    else:
        dys, lddys = _rows_out(out, R, H, ys)
    dw = torch.empty((T, k), dtype=torch.float32, device=dy.device)
    status = (_lib or lib()).fp8_moe_combine_grad(dy.data_ptr(), f32, T, H, lddy, ys.data_ptr(), R, ldys,
                                                  pos.data_ptr(), weights.data_ptr(), k, dys.data_ptr(), lddys,
                                                  dw.data_ptr(), _stream_ptr(dy))
    if status:
        raise FP8Error(status, "fp8_moe_combine_grad")
    return dys, dw


def fp8_moe_dispatch_grad(dxs, pos, out=None):
    """The gradient of fp8_moe_dispatch: dx[t] = sum_j dxs[pos[t, j]]."""
    f32, R, H, lddxs = _check_rows_in(dxs, "dxs")
    T, k = _check_pairs(pos, None, dxs.get_device())
    dx, lddx = _rows_out(out, T, H, dxs)
    status = (_lib or lib()).fp8_moe_dispatch_grad(dxs.data_ptr(), f32, R, H, lddxs, pos.data_ptr(), T, k,
                                                   dx.data_ptr(), lddx, _stream_ptr(dxs))
    if status:
        raise FP8Error(status, "fp8_moe_dispatch_grad")
    return dx


# ---------------------------------------------------------------------------
# norms around a block
# ---------------------------------------------------------------------------

def _norm_operands(torch, y, weight, residual, post_weight, gate, scale, residual_out):
    """Checks what both norms share; (M, H, ldy, index, gate's row stride, residual's, r, r's row stride). r is None
    where nothing changes y."""
    if y.dtype is not torch.bfloat16 or y.dim() != 2 or not y.is_cuda:
        raise ValueError("y: expected a CUDA bf16 matrix with unit column stride")
    M, H = y.shape
    ldy, unit = y.stride()
    if unit != 1 and H > 1:
        raise ValueError("y: expected a CUDA bf16 matrix with unit column stride")
    index = y.get_device()
    if weight is not None:
        _check_dense(weight, torch.bfloat16, (H,), index, "weight")
    if post_weight is not None:
        _check_dense(post_weight, torch.bfloat16, (H,), index, "post_weight")
    ldg = 0
    if gate is not None:
        if gate.dim() == 1:
            _check_dense(gate, torch.bfloat16, (H,), index, "gate")
        else:
            _check_rows(gate, torch.bfloat16, M, H, index, "gate")
            ldg = _row_stride(gate, M, H)
    ldr = 0
    if residual is not None:
        _check_rows(residual, torch.bfloat16, M, H, index, "residual")
        ldr = _row_stride(residual, M, H)
    if residual_out is not None:
        r = _out_bf16(residual_out, M, H, y)
        ldro = _row_stride(r, M, H)
    elif residual is None and post_weight is None and gate is None and scale == 1.0:
        r, ldro = None, 0
    else:
        r, ldro = torch.empty((M, H), dtype=torch.bfloat16, device=y.device), H or 1
    return M, H, ldy if M > 1 else H or 1, index, ldg, ldr, r, ldro


def fp8_residual_norm(y, weight=None, residual=None, post_weight=None, gate=None, scale: float = 1.0,
                      eps: float = 1e-6, plus_one: bool = False, out=None, residual_out=None):
    """The end of a block and the norm before the next: (n, r) bf16 [M, H] of y bf16 [M, H], with
    t = y (with post_weight: y / sqrt(mean y^2 + eps) * post_weight), r = residual + scale * gate * t and
    n = r / sqrt(mean r^2 + eps) * weight, in fp32 with one rounding of r and of n. Weights bf16 [H] (plus_one: they
    stand for 1 + weight), gate bf16 [H] or [M, H]. Without a weight n is None; where nothing changes y, r is y, or None if
    n took y's place (out is y). residual_out may be y or residual itself."""
    torch = _torch_module or _torch()
    M, H, ldy, index, ldg, ldr, r, ldro = _norm_operands(torch, y, weight, residual, post_weight, gate, scale,
                                                         residual_out)
    n = None
    if weight is not None:
        n = torch.empty((M, H), dtype=torch.bfloat16, device=y.device) if out is None else _out_bf16(out, M, H, y)
    elif out is not None:
        raise ValueError("out: there is no n without a weight")
    if n is None and r is None:
        return None, y
    status = (_lib or lib()).fp8_residual_norm(
        y.data_ptr(), M, H, ldy, _ptr(post_weight), _ptr(gate), ldg, scale, _ptr(residual), ldr, _ptr(weight), eps,
        1 if plus_one else 0, _ptr(r), ldro, _ptr(n), 0 if n is None else _row_stride(n, M, H), _stream_ptr(y))
    if status:
        raise FP8Error(status, "fp8_residual_norm")
    if r is None and (out is None or out.data_ptr() != y.data_ptr() or not M * H):
        r = y
    return n, r


def fp8_residual_norm_quantize(y, weight, residual=None, post_weight=None, gate=None, scale: float = 1.0,
                               eps: float = 1e-6, plus_one: bool = False, residual_out=None):
    """fp8_residual_norm with n quantized for fp8_block_scaled_mm: (qn uint8 [M, min_ld(H)], s_n fp32
    [ceil(H/128), M], r), one scale per row and 128 columns, as fp8_block_quantize_act returns them."""
    torch = _torch_module or _torch()
    M, H, ldy, index, ldg, ldr, r, ldro = _norm_operands(torch, y, weight, residual, post_weight, gate, scale,
                                                         residual_out)
    if weight is None:
        raise ValueError("weight: expected a bf16 vector")
    ldq, device = min_ld(H), y.device
    lds = (M + 3) // 4 * 4 or 1
    qn = torch.empty((M, ldq), dtype=torch.uint8, device=device)
    # the last row ends with its last scale, within the 16 bytes that a copy of whole pieces reads
    s_n = torch.empty_strided((_blocks(H), M), (lds, 1), dtype=torch.float32, device=device)
    status = (_lib or lib()).fp8_residual_norm_quantize(
        y.data_ptr(), M, H, ldy, _ptr(post_weight), _ptr(gate), ldg, scale, _ptr(residual), ldr, weight.data_ptr(), eps,
        1 if plus_one else 0, _ptr(r), ldro, qn.data_ptr(), ldq, s_n.data_ptr(), lds, _stream_ptr(y))
    if status:
        raise FP8Error(status, "fp8_residual_norm_quantize")
    return qn, s_n, y if r is None else r


def fp8_selftest_timeout(limit_ns: int = 20_000_000, stream=None) -> int:
    """Enqueue the failure-path self-test (a bounded device wait made to run out); returns the status."""
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream().cuda_stream
    return int(lib().fp8_selftest_timeout(int(limit_ns), s))


def fp8_block_selftest_timeout(form: int, qa, K: int, s_a, qw, s_w, out, s_out=None, stream=None) -> int:
    """Enqueue the block-scaled product with one load withheld from its waits (forms: see the C header); returns
    the status."""
    if stream is None:
        stream = _torch().cuda.current_stream().cuda_stream
    return int(lib().fp8_block_selftest_timeout(
        form, qa.data_ptr(), qa.shape[0], K, qa.stride(0), s_a.data_ptr(), s_a.stride(0), qw.data_ptr(), qw.shape[-2],
        qw.shape[-1], s_w.data_ptr(), out.data_ptr(), out.stride(0), _ptr(s_out),
        0 if s_out is None else s_out.stride(0), stream))


def fp8_lora_selftest_timeout(form: int, y, x, a, b, ids, scales, out, ws, stream=None) -> int:
    """Enqueue fp8_lora_add with one load withheld from its waits (forms: see the C header); returns the status."""
    if stream is None:
        stream = _torch().cuda.current_stream().cuda_stream
    return int(lib().fp8_lora_selftest_timeout(
        form, y.data_ptr(), y.shape[0], y.shape[1], y.stride(0), x.data_ptr(), x.shape[1], x.stride(0), a.data_ptr(),
        b.data_ptr(), a.shape[0], a.shape[1], ids.data_ptr(), _ptr(scales), out.data_ptr(), out.stride(0), ws.data_ptr(),
        ws.numel(), stream))


def fp8_last_device_status(stream=None) -> int:
    """Synchronizes the stream; returns FP8_OK or the device-side error the kernels recorded."""
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream().cuda_stream
    return int(lib().fp8_last_device_status(s))


def fp8_gemm_config(qa, qw, K: Optional[int] = None, ws_bytes: int = 0) -> dict:
    """The GEMM launch the library would use for FP8 operands qa [M, ld] and qw [N, ld] (K columns;
    default: the row length) with a linear workspace of ws_bytes, on the current device:
    {"two_sm": bool, "grid": int, "group_n": int, "splits": int, "tail_split": int}. Enqueues nothing."""
    two, grid, gn, sp, ts = (ctypes.c_int(0) for _ in range(5))
    K = qa.shape[1] if K is None else int(K)
    st = lib().fp8_gemm_config(qa.data_ptr(), qa.shape[0], qa.stride(0), qw.data_ptr(), qw.shape[0], qw.stride(0),
                               K, int(ws_bytes), ctypes.byref(two), ctypes.byref(grid), ctypes.byref(gn),
                               ctypes.byref(sp), ctypes.byref(ts))
    if st != FP8_OK:
        raise FP8Error(st, "fp8_gemm_config")
    return {"two_sm": bool(two.value), "grid": grid.value, "group_n": gn.value, "splits": sp.value,
            "tail_split": ts.value}


def fp8_gemm_plan_model(M: int, N: int, K: int, num_sms: int = 152, pair_slots: int = 76, ws_bytes: int = 0) -> dict:
    """The GEMM launch plan fp8_gemm_config would report for gap-free FP8 operands in a GPU's own
    memory, computed on the host (no device): same keys."""
    two, grid, gn, sp, ts = (ctypes.c_int(0) for _ in range(5))
    st = lib().fp8_gemm_plan_model(int(M), int(N), int(K), int(num_sms), int(pair_slots), int(ws_bytes),
                                   ctypes.byref(two), ctypes.byref(grid), ctypes.byref(gn), ctypes.byref(sp),
                                   ctypes.byref(ts))
    if st != FP8_OK:
        raise FP8Error(st, "fp8_gemm_plan_model")
    return {"two_sm": bool(two.value), "grid": grid.value, "group_n": gn.value, "splits": sp.value,
            "tail_split": ts.value}


def fp8_gemv_plan_model(M: int, N: int, K: int, mode: int, clusters_of_size, smem_limit: int = 227 * 1024,
                        static_scale: bool = False) -> dict:
    """The decode GEMV's launch configuration computed on the host (no device): mode 0 activations
    pre-quantized, 1 quantized in the kernel, 2 bf16 (weight-only); clusters_of_size[s - 1] =
    co-resident clusters of s CTAs, s = 1..8."""
    occ = (ctypes.c_int * 8)(*[int(x) for x in clusters_of_size])
    outs = [ctypes.c_int(0) for _ in range(7)]
    st = lib().fp8_gemv_plan_model(int(M), int(N), int(K), int(mode), int(bool(static_scale)), int(smem_limit),
                                   ctypes.cast(occ, ctypes.c_void_p), *[ctypes.byref(o) for o in outs])
    if st != FP8_OK:
        raise FP8Error(st, "fp8_gemv_plan_model")
    keys = ("cluster", "clusters", "stages", "kslice", "scratch_a", "cluster_amax", "tcgen05")
    return {k: o.value for k, o in zip(keys, outs)}


def min_workspace_bytes(M: int, K: int, N: int) -> int:
    """The least workspace fp8_linear accepts for this shape (no K split): 0 for decode shapes of
    up to 16 tokens, which the GEMV quantizes itself."""
    if M <= 0 or K <= 0 or (M <= 16 and fp8_uses_gemv(M, K, N)):
        return 0
    return FP8_QUANT_WORKSPACE_BYTES + M * min_ld(K)
