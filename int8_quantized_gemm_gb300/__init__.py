"""GB300 W8A8 quantized linear layer: Python binding of the C ABI in include/q8.h.

Argument marshalling only: every step of the path runs in the CUDA kernels of
libq8.so. PyTorch supplies device memory and the current stream. There is no
CPU fallback; if the library is missing or a call fails, an exception says so.

  q8_quantize_act(a, per_row=True, symmetric=True)   -> qa, s_a, z_a
  q8_rmsnorm_quantize_act(a, gamma, eps)             -> qa, s_a   (fused RMSNorm + per-token quantize)
  q8_quantize_weight(w, per_row=True)                 -> qw, s_w
  q8_colsum(qw)                                       -> colsum
  q8_gemm_dequant(qa, s_a, z_a, qw, s_w, colsum)      -> y
  q8_gemm_epilogue(qa, s_a, z_a, qw, s_w, colsum, bias, out_dtype, out_scale) -> y (+bias; fp32/bf16/int8)
  q8_gemm_s32(qa, qw)                                 -> acc (raw INT32 accumulators)
  q8_quantize_weight_int4(w) -> qw4, s_w;  q8_colsum_int4(qw4, K);  q8_gemm_w4a8(qa, s_a, z_a, qw4, s_w, ...)
  q8_quantize_weight_mx(w, group) -> qw, sf;  q8_gemm_mx(qa, s_a, qw, sf, group, ...)   (block-scaled weights)
  q8_linear(a, qw, s_w, colsum)                       -> y   (quantize A, then GEMM)
  q8_linear_host(a_host, qw, s_w, colsum, y_host)      (host buffers; copies overlapped with the device work)

Float8 (e4m3) operands with a scale for each block of 128, and layers of routed experts:

  q8_quantize_fp8(x, slots=None)          -> qa, sa    (or each row to the slots of its experts)
  q8_swiglu_quantize_fp8(h)               -> qa, sa    (gated activation + quantize)
  q8_quantize_weight_fp8(w)               -> qw, sw    ([N, K] or [E, N, K])
  q8_gemm_fp8(qa, sa, qw, sw)             -> y
  q8_gemm_fp8_grouped(qa, sa, qw, sw, offsets) -> y    (row ranges of experts)
  q8_moe_route(logits, top_k, ...)        -> idx, weights
  q8_moe_plan(idx, n_experts)             -> offsets, slots
  q8_moe_combine(h, slots, weights)       -> y

4-bit floating point (e2m1) operands with a scale for each block of 16 (e4m3, under one fp32 scale a row) or 32 K (a power of two):

  q8_quantize_fp4(x, block=16, slots=None)      -> q, sf, s     (s is None for block 32)
  q8_swiglu_quantize_fp4(h, block=16)           -> q, sf, s     (gated activation + quantize)
  q8_quantize_weight_fp4(w, block=16)           -> qw, sfw, sw  ([N, K] or [E, N, K]; scales in the tensor core's order)
  q8_dequantize_fp4(q, sf, s)                   -> y            (what the codes stand for)
  q8_gemm_fp4(qa, sfa, sa, qw, sfw, sw)         -> y
  q8_gemm_fp4_grouped(qa, sfa, sa, qw, sfw, sw, offsets) -> y   (row ranges of experts)
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import warnings

import torch

from . import build as _build

__all__ = [
    "Q8Error", "load", "q8_quantize_act", "q8_rmsnorm_quantize_act", "q8_quantize_weight", "q8_colsum", "q8_gemm_dequant",
    "q8_gemm_epilogue", "q8_gemm_s32", "q8_linear", "q8_quantize_weight_int4", "q8_colsum_int4", "q8_gemm_w4a8",
    "q8_gemm_w4a8_s32", "q8_quantize_weight_mx", "q8_gemm_mx", "q8_quantize_act_f16", "q8_quantize_act_dual", "q8_gemm_f16a", "q8_gemm_f16a_s32", "q8_linear_host", "q8_linear_host_workspace", "q8_gemm_workspace", "q8_gemm_pick", "q8_launch_count", "q8_device_error",
    "q8_selftest_wait_timeout", "KERNELS", "q8_quantize_fp8", "q8_swiglu_quantize_fp8", "q8_quantize_weight_fp8",
    "q8_gemm_fp8", "q8_gemm_fp8_grouped", "q8_moe_route", "q8_moe_plan", "q8_moe_combine", "q8_quantize_fp4",
    "q8_swiglu_quantize_fp4", "q8_quantize_weight_fp4", "q8_dequantize_fp4", "q8_gemm_fp4", "q8_gemm_fp4_grouped",
]

LIB_PATH = _build.LIB
Q8_OK, Q8_ERR_INVALID_ARG, Q8_ERR_UNSUPPORTED, Q8_ERR_CUDA, Q8_ERR_TIMEOUT = range(5)
Q8_PER_TENSOR, Q8_PER_ROW = 0, 1
Q8_SYMMETRIC, Q8_ASYMMETRIC = 0, 1
KERNELS = {"auto": 0, "tcgen05": 1, "mma_s8": 2, "skinny": 3, "decode": 4, "decode_tc": 5, "tcgen05_pair": 6}
KERNEL_NAMES = {v: k for k, v in KERNELS.items()}

_lib = None
_calls = None   # the common calls of the 4-bit operators (csrc/q8_calls.cpp); None: the binding makes them itself


class Q8Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libq8.so (built in-tree by build.py). Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"libq8.so is not built ({path}); run int8_quantized_gemm_gb300.build.build()")
    lib = ctypes.CDLL(path)
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.q8_quantize_act.argtypes = [p, i64, i64, i32, i32, p, p, p, p]
    lib.q8_rmsnorm_quantize_act.argtypes = [p, p, i64, i64, ctypes.c_float, p, p, p]
    lib.q8_quantize_weight.argtypes = [p, i64, i64, i32, p, p, p]
    lib.q8_colsum.argtypes = [p, i64, i64, p, p]
    lib.q8_gemm_dequant.argtypes = [p, p, p, i32, p, p, i32, p, i64, i64, i64, p, p]
    lib.q8_gemm_dequant_ex.argtypes = [p, p, p, i32, p, p, i32, p, i64, i64, i64, p, i32, p]
    lib.q8_gemm_dequant_ws.argtypes = [p, p, p, i32, p, p, i32, p, i64, i64, i64, p, p, ctypes.c_size_t, p]
    lib.q8_gemm_workspace.argtypes = [i64, i64, i64]
    lib.q8_gemm_workspace.restype = ctypes.c_size_t
    lib.q8_gemm_epilogue_ex.argtypes = [p, p, p, i32, p, p, i32, p, p, i64, i64, i64, i32, p, ctypes.c_float, i32, p]
    lib.q8_gemm_s32_ex.argtypes = [p, p, i64, i64, i64, p, i32, p]
    lib.q8_quantize_act_f16.argtypes = [p, i64, i64, i32, i32, p, p, p, p]
    lib.q8_gemm_f16a_ex.argtypes = [p, p, p, i32, p, p, i32, p, p, i64, i64, i64, i32, p, ctypes.c_float, p]
    lib.q8_gemm_f16a_s32.argtypes = [p, p, i64, i64, i64, p, p]
    lib.q8_quantize_weight_int4.argtypes = [p, i64, i64, p, p, p]
    lib.q8_colsum_int4.argtypes = [p, i64, i64, p, p]
    lib.q8_gemm_w4a8_ex.argtypes = [p, p, p, i32, p, p, p, p, i64, i64, i64, i32, p, ctypes.c_float, i32, p]
    lib.q8_gemm_w4a8_s32_ex.argtypes = [p, p, i64, i64, i64, p, i32, p]
    lib.q8_quantize_weight_mx.argtypes = [p, i64, i64, i32, p, p, p]
    lib.q8_gemm_mx_ex.argtypes = [p, p, i32, p, p, i32, p, i64, i64, i64, i32, p, ctypes.c_float, i32, p]
    lib.q8_gemm_w4a8_ws.argtypes = [p, p, p, i32, p, p, p, p, i64, i64, i64, i32, p, ctypes.c_float, p,
                                    ctypes.c_size_t, p]
    lib.q8_gemm_mx_ws.argtypes = [p, p, i32, p, p, i32, p, i64, i64, i64, i32, p, ctypes.c_float, p,
                                  ctypes.c_size_t, p]
    lib.q8_linear.argtypes = [p, i64, i64, i32, i32, p, p, p, p, p, i32, p, i64, p, p]
    lib.q8_linear_ws.argtypes = [p, i64, i64, i32, i32, p, p, p, p, p, i32, p, i64, p, p, ctypes.c_size_t, p]
    lib.q8_quantize_act_dual.argtypes = [p, i64, i64, i32, i32, p, p, p, p, p]
    lib.q8_selftest_wait_timeout.argtypes = [i32, p, p, i64, i64, i64, p, i64, p]
    lib.q8_linear_host_workspace.argtypes = [i64, i64, i64, i64]
    lib.q8_linear_host_workspace.restype = ctypes.c_size_t
    lib.q8_linear_host.argtypes = [p, i64, i64, i32, p, p, i32, p, i64, p, i64, p, ctypes.c_size_t, p]
    lib.q8_gemm_pick.argtypes = [i64, i64, i64]
    lib.q8_status_string.argtypes = [i32]
    lib.q8_status_string.restype = ctypes.c_char_p
    lib.q8_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    lib.q8_launch_count.argtypes = []
    lib.q8_launch_count.restype = ctypes.c_uint64
    lib.q8_quantize_fp8.argtypes = [p, i32, i64, i64, i64, p, i64, i64, p, p, p]
    lib.q8_swiglu_quantize_fp8.argtypes = [p, i32, i64, i64, i64, p, p, p]
    lib.q8_quantize_weight_fp8.argtypes = [p, i32, i64, i64, i64, p, p, p]
    lib.q8_gemm_fp8.argtypes = [p, p, p, p, i64, i64, i64, p, i32, p]
    lib.q8_gemm_fp8_grouped.argtypes = [p, p, p, p, p, i64, i64, i64, i64, p, i32, p]
    lib.q8_moe_route.argtypes = [p, i32, i64, i64, i64, i64, i32, p, i64, i64, i32, ctypes.c_float, p, p, p]
    lib.q8_moe_plan.argtypes = [p, i64, i64, i64, p, p, p]
    lib.q8_moe_combine.argtypes = [p, i32, i64, i64, p, p, i64, i64, p, p]
    lib.q8_quantize_fp4.argtypes = [p, i32, i32, i64, i64, i64, p, i64, i64, p, p, p, p]
    lib.q8_swiglu_quantize_fp4.argtypes = [p, i32, i32, i64, i64, i64, p, p, p, p]
    lib.q8_quantize_weight_fp4.argtypes = [p, i32, i32, i64, i64, i64, p, p, p, p]
    lib.q8_dequantize_fp4.argtypes = [p, p, p, i32, i64, i64, i64, p, i32, p]
    lib.q8_gemm_fp4.argtypes = [p, p, p, p, p, p, i32, i64, i64, i64, p, i32, p]
    lib.q8_gemm_fp4_grouped.argtypes = [p, p, p, p, p, p, p, i32, i64, i64, i64, i64, p, i32, p]
    for name in ("q8_quantize_fp4", "q8_swiglu_quantize_fp4", "q8_quantize_weight_fp4", "q8_dequantize_fp4", "q8_gemm_fp4",
                 "q8_gemm_fp4_grouped", "q8_quantize_fp8", "q8_swiglu_quantize_fp8", "q8_quantize_weight_fp8", "q8_gemm_fp8",
                 "q8_gemm_fp8_grouped", "q8_moe_route", "q8_moe_plan", "q8_moe_combine",
                 "q8_quantize_act", "q8_rmsnorm_quantize_act", "q8_quantize_weight", "q8_colsum", "q8_gemm_dequant",
                 "q8_gemm_dequant_ex", "q8_gemm_dequant_ws", "q8_gemm_epilogue_ex", "q8_gemm_s32_ex", "q8_quantize_weight_int4",
                 "q8_colsum_int4", "q8_gemm_w4a8_ex", "q8_gemm_w4a8_s32_ex", "q8_quantize_weight_mx", "q8_gemm_mx_ex",
                 "q8_gemm_w4a8_ws", "q8_gemm_mx_ws", "q8_linear_ws", "q8_quantize_act_dual",
                 "q8_linear", "q8_linear_host", "q8_gemm_pick", "q8_device_error", "q8_selftest_wait_timeout"):
        getattr(lib, name).restype = i32
    _lib = lib
    _load_calls(lib)
    return lib


def _load_calls(lib: ctypes.CDLL):
    """The module of the common calls, where it is built. One that does not load (built against another PyTorch, say) is reported
    and not used: the binding makes the same calls."""
    global _calls
    path = _build.calls_path()
    if not os.path.exists(path):
        return
    try:
        loader = importlib.machinery.ExtensionFileLoader("_q8_calls", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_q8_calls", loader))
        loader.exec_module(module)
        module.entries(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                         for name in ("q8_quantize_fp4", "q8_swiglu_quantize_fp4", "q8_dequantize_fp4", "q8_gemm_fp4",
                                      "q8_gemm_fp4_grouped")))
    except Exception as e:      # whatever it is, no call depends on this module
        warnings.warn(f"{path} does not load, the binding makes its calls itself: {e}", RuntimeWarning, stacklevel=3)
        return
    _calls = module


def status_string(status: int) -> str:
    return load().q8_status_string(status).decode()


def _check(status: int, what: str):
    if status != Q8_OK:
        raise Q8Error(status, what)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t: torch.Tensor, dtype, name: str, ndim: int | None = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


def q8_quantize_act(a: torch.Tensor, per_row: bool = True, symmetric: bool = True, qa=None, s_a=None,
                    z_a=None, stream=None):
    """Dynamic activation quantization of fp32 a[M, K]; returns (qa int8, s_a fp32, z_a int32 or None)."""
    _need(a, torch.float32, "a", 2)
    M, K = a.shape
    n = M if per_row else 1
    qa = torch.empty((M, K), dtype=torch.int8, device=a.device) if qa is None else qa
    s_a = torch.empty(n, dtype=torch.float32, device=a.device) if s_a is None else s_a
    if not symmetric and z_a is None:
        z_a = torch.empty(n, dtype=torch.int32, device=a.device)
    if symmetric:
        z_a = None
    _check(load().q8_quantize_act(_ptr(a), M, K, Q8_PER_ROW if per_row else Q8_PER_TENSOR,
                                  Q8_SYMMETRIC if symmetric else Q8_ASYMMETRIC, _ptr(qa), _ptr(s_a),
                                  _ptr(z_a), _stream(stream)), "q8_quantize_act")
    return qa, s_a, z_a


def q8_rmsnorm_quantize_act(a: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6, qa=None, s_a=None,
                            stream=None):
    """Fused RMSNorm (weights gamma[K], eps under the root) + per-token symmetric quantization
    of fp32 a[M, K]; returns (qa int8 [M, K], s_a fp32 [M])."""
    _need(a, torch.float32, "a", 2)
    _need(gamma, torch.float32, "gamma", 1)
    M, K = a.shape
    if gamma.numel() != K:
        raise ValueError("gamma must have K entries")
    qa = torch.empty((M, K), dtype=torch.int8, device=a.device) if qa is None else qa
    s_a = torch.empty(M, dtype=torch.float32, device=a.device) if s_a is None else s_a
    _check(load().q8_rmsnorm_quantize_act(_ptr(a), _ptr(gamma), M, K, ctypes.c_float(eps), _ptr(qa), _ptr(s_a),
                                          _stream(stream)), "q8_rmsnorm_quantize_act")
    return qa, s_a


def q8_quantize_weight(w: torch.Tensor, per_row: bool = True, qw=None, s_w=None, stream=None):
    """Symmetric quantization of fp32 W[N, K] (K-major); returns (qw int8, s_w fp32)."""
    _need(w, torch.float32, "w", 2)
    N, K = w.shape
    qw = torch.empty((N, K), dtype=torch.int8, device=w.device) if qw is None else qw
    s_w = torch.empty(N if per_row else 1, dtype=torch.float32, device=w.device) if s_w is None else s_w
    _check(load().q8_quantize_weight(_ptr(w), N, K, Q8_PER_ROW if per_row else Q8_PER_TENSOR, _ptr(qw),
                                     _ptr(s_w), _stream(stream)), "q8_quantize_weight")
    return qw, s_w


def q8_colsum(qw: torch.Tensor, out=None, stream=None):
    _need(qw, torch.int8, "qw", 2)
    N, K = qw.shape
    out = torch.empty(N, dtype=torch.int32, device=qw.device) if out is None else out
    _check(load().q8_colsum(_ptr(qw), N, K, _ptr(out), _stream(stream)), "q8_colsum")
    return out


def q8_gemm_workspace(M: int, N: int, K: int) -> int:
    """Device workspace bytes q8_gemm_dequant(..., workspace=) can use for this shape (0: none)."""
    return int(load().q8_gemm_workspace(M, N, K))


def q8_gemm_dequant(qa, s_a, z_a, qw, s_w, colsum=None, y=None, kernel: str = "auto", workspace=None,
                    stream=None):
    """y[M, N] = (acc - z_a*colsum) * (s_a * s_w) from int8 codes; per-row scales are inferred
    from the lengths of s_a (M entries) and s_w (N entries). workspace: an optional device tensor of
    at least q8_gemm_workspace(M, N, K) bytes (kernel "auto" only; q8_gemm_dequant_ws)."""
    _need(qa, torch.int8, "qa", 2)
    _need(qw, torch.int8, "qw", 2)
    M, K = qa.shape
    N = qw.shape[0]
    if qw.shape[1] != K:
        raise ValueError("qa and qw disagree on K")
    _need(s_a, torch.float32, "s_a", 1)
    _need(s_w, torch.float32, "s_w", 1)
    ga = Q8_PER_ROW if (s_a.numel() == M and M != 1) else Q8_PER_TENSOR
    gw = Q8_PER_ROW if (s_w.numel() == N and N != 1) else Q8_PER_TENSOR
    if s_a.numel() not in (1, M) or s_w.numel() not in (1, N):
        raise ValueError("s_a must have 1 or M entries and s_w 1 or N entries")
    if z_a is not None:
        _need(z_a, torch.int32, "z_a", 1)
        if z_a.numel() != s_a.numel():
            raise ValueError("z_a must have as many entries as s_a")
        if colsum is None:
            raise ValueError("an asymmetric A needs the weight column sums")
        _need(colsum, torch.int32, "colsum", 1)
    y = torch.empty((M, N), dtype=torch.float32, device=qa.device) if y is None else y
    _need(y, torch.float32, "y", 2)
    if workspace is not None:
        if kernel != "auto":
            raise ValueError("a workspace goes with the automatic kernel choice")
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        _check(load().q8_gemm_dequant_ws(_ptr(qa), _ptr(s_a), _ptr(z_a), ga, _ptr(qw), _ptr(s_w), gw,
                                         _ptr(colsum if z_a is not None else None), M, N, K, _ptr(y),
                                         _ptr(workspace), workspace.numel() * workspace.element_size(),
                                         _stream(stream)), "q8_gemm_dequant_ws")
        return y
    _check(load().q8_gemm_dequant_ex(_ptr(qa), _ptr(s_a), _ptr(z_a), ga, _ptr(qw), _ptr(s_w), gw,
                                     _ptr(colsum if z_a is not None else None), M, N, K, _ptr(y),
                                     KERNELS[kernel], _stream(stream)), "q8_gemm_dequant")
    return y


OUT_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.int8: 2}


def _epilogue_args(qa, qa_dtype, s_a, z_a, qw, s_w, colsum, bias, out_dtype, out_scale, out):
    """Checks of the epilogue entries; returns (M, N, K, ga, gw, out)."""
    _need(qa, qa_dtype, "qa", 2)
    _need(qw, torch.int8, "qw", 2)
    M, K = qa.shape
    N = qw.shape[0]
    if qw.shape[1] != K:
        raise ValueError("qa and qw disagree on K")
    if out_dtype not in OUT_TYPES:
        raise TypeError("out_dtype must be torch.float32, torch.bfloat16 or torch.int8")
    _need(s_a, torch.float32, "s_a", 1)
    _need(s_w, torch.float32, "s_w", 1)
    if s_a.numel() not in (1, M) or s_w.numel() not in (1, N):
        raise ValueError("s_a must have 1 or M entries and s_w 1 or N entries")
    ga = Q8_PER_ROW if (s_a.numel() == M and M != 1) else Q8_PER_TENSOR
    gw = Q8_PER_ROW if (s_w.numel() == N and N != 1) else Q8_PER_TENSOR
    if z_a is not None:
        _need(z_a, torch.int32, "z_a", 1)
        if colsum is None:
            raise ValueError("an asymmetric A needs the weight column sums")
        _need(colsum, torch.int32, "colsum", 1)
    if bias is not None:
        _need(bias, torch.float32, "bias", 1)
        if bias.numel() != N:
            raise ValueError("bias must have N entries")
    if out_dtype == torch.int8 and out_scale is None:
        raise ValueError("int8 output needs out_scale")
    out = torch.empty((M, N), dtype=out_dtype, device=qa.device) if out is None else out
    _need(out, out_dtype, "out", 2)
    return M, N, K, ga, gw, out


def q8_quantize_act_f16(a: torch.Tensor, per_row: bool = True, symmetric: bool = True, qa16=None, s_a=None,
                        z_a=None, stream=None):
    """q8_quantize_act with the codes written as fp16 values; returns (qa16 float16, s_a, z_a or None)."""
    _need(a, torch.float32, "a", 2)
    M, K = a.shape
    n = M if per_row else 1
    qa16 = torch.empty((M, K), dtype=torch.float16, device=a.device) if qa16 is None else qa16
    _need(qa16, torch.float16, "qa16", 2)
    s_a = torch.empty(n, dtype=torch.float32, device=a.device) if s_a is None else s_a
    if not symmetric and z_a is None:
        z_a = torch.empty(n, dtype=torch.int32, device=a.device)
    if symmetric:
        z_a = None
    _check(load().q8_quantize_act_f16(_ptr(a), M, K, Q8_PER_ROW if per_row else Q8_PER_TENSOR,
                                      Q8_SYMMETRIC if symmetric else Q8_ASYMMETRIC, _ptr(qa16), _ptr(s_a),
                                      _ptr(z_a), _stream(stream)), "q8_quantize_act_f16")
    return qa16, s_a, z_a


def q8_quantize_act_dual(a: torch.Tensor, per_row: bool = True, symmetric: bool = True, qa=None, qa16=None,
                         s_a=None, z_a=None, stream=None):
    """q8_quantize_act that also writes the codes as fp16 values (for q8_gemm_f16a); returns
    (qa int8, qa16 float16, s_a, z_a or None)."""
    _need(a, torch.float32, "a", 2)
    M, K = a.shape
    n = M if per_row else 1
    qa = torch.empty((M, K), dtype=torch.int8, device=a.device) if qa is None else qa
    qa16 = torch.empty((M, K), dtype=torch.float16, device=a.device) if qa16 is None else qa16
    _need(qa16, torch.float16, "qa16", 2)
    s_a = torch.empty(n, dtype=torch.float32, device=a.device) if s_a is None else s_a
    if not symmetric and z_a is None:
        z_a = torch.empty(n, dtype=torch.int32, device=a.device)
    if symmetric:
        z_a = None
    _check(load().q8_quantize_act_dual(_ptr(a), M, K, Q8_PER_ROW if per_row else Q8_PER_TENSOR,
                                       Q8_SYMMETRIC if symmetric else Q8_ASYMMETRIC, _ptr(qa), _ptr(qa16), _ptr(s_a),
                                       _ptr(z_a), _stream(stream)), "q8_quantize_act_dual")
    return qa, qa16, s_a, z_a


def q8_gemm_f16a(qa16, s_a, z_a, qw, s_w, colsum=None, bias=None, out_dtype=torch.float32, out_scale=None,
                 out=None, stream=None):
    """q8_gemm_epilogue on fp16-valued activation codes (from q8_quantize_act_f16)."""
    M, N, K, ga, gw, out = _epilogue_args(qa16, torch.float16, s_a, z_a, qw, s_w, colsum, bias, out_dtype,
                                          out_scale, out)
    _check(load().q8_gemm_f16a_ex(_ptr(qa16), _ptr(s_a), _ptr(z_a), ga, _ptr(qw), _ptr(s_w), gw,
                                  _ptr(colsum if z_a is not None else None), _ptr(bias), M, N, K,
                                  OUT_TYPES[out_dtype], _ptr(out), ctypes.c_float(out_scale or 0.0),
                                  _stream(stream)), "q8_gemm_f16a")
    return out


def q8_gemm_f16a_s32(qa16, qw, out=None, stream=None):
    """Raw INT32 accumulators of q8_gemm_f16a."""
    _need(qa16, torch.float16, "qa16", 2)
    _need(qw, torch.int8, "qw", 2)
    M, K = qa16.shape
    N = qw.shape[0]
    if qw.shape[1] != K:
        raise ValueError("qa16 and qw disagree on K")
    out = torch.empty((M, N), dtype=torch.int32, device=qa16.device) if out is None else out
    _need(out, torch.int32, "out", 2)
    _check(load().q8_gemm_f16a_s32(_ptr(qa16), _ptr(qw), M, N, K, _ptr(out), _stream(stream)), "q8_gemm_f16a_s32")
    return out


def q8_gemm_epilogue(qa, s_a, z_a, qw, s_w, colsum=None, bias=None, out_dtype=torch.float32, out_scale=None,
                     out=None, kernel: str = "auto", stream=None):
    """Quantized linear layer with the epilogue variants: y = (acc - z_a*colsum) * (s_a*s_w) + bias,
    written as fp32, bf16, or int8 codes with the static output scale out_scale."""
    M, N, K, ga, gw, out = _epilogue_args(qa, torch.int8, s_a, z_a, qw, s_w, colsum, bias, out_dtype, out_scale,
                                          out)
    _check(load().q8_gemm_epilogue_ex(_ptr(qa), _ptr(s_a), _ptr(z_a), ga, _ptr(qw), _ptr(s_w), gw,
                                      _ptr(colsum if z_a is not None else None), _ptr(bias), M, N, K,
                                      OUT_TYPES[out_dtype], _ptr(out), ctypes.c_float(out_scale or 0.0),
                                      KERNELS[kernel], _stream(stream)), "q8_gemm_epilogue")
    return out


def q8_quantize_weight_int4(w: torch.Tensor, qw4=None, s_w=None, stream=None):
    """Per-channel symmetric int4 codes of fp32 W[N, K], packed two per byte: (qw4 uint8 [N, K/2], s_w [N])."""
    _need(w, torch.float32, "w", 2)
    N, K = w.shape
    qw4 = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device) if qw4 is None else qw4
    s_w = torch.empty(N, dtype=torch.float32, device=w.device) if s_w is None else s_w
    _check(load().q8_quantize_weight_int4(_ptr(w), N, K, _ptr(qw4), _ptr(s_w), _stream(stream)),
           "q8_quantize_weight_int4")
    return qw4, s_w


def q8_colsum_int4(qw4: torch.Tensor, K: int, out=None, stream=None):
    _need(qw4, torch.uint8, "qw4", 2)
    N = qw4.shape[0]
    if qw4.shape[1] * 2 != K:
        raise ValueError("qw4 must be [N, K / 2]")
    out = torch.empty(N, dtype=torch.int32, device=qw4.device) if out is None else out
    _check(load().q8_colsum_int4(_ptr(qw4), N, K, _ptr(out), _stream(stream)), "q8_colsum_int4")
    return out


def _ws_args(workspace, kernel):
    if kernel != "auto":
        raise ValueError("a workspace goes with the automatic kernel choice")
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def q8_gemm_w4a8(qa, s_a, z_a, qw4, s_w, colsum=None, bias=None, out_dtype=torch.float32, out_scale=None,
                 out=None, kernel: str = "auto", workspace=None, stream=None):
    """W4A8 linear layer: int8 activations x packed int4 weights, epilogue as q8_gemm_epilogue.
    workspace: an optional device tensor of at least 2 M K bytes for the fp16 copy of the codes
    (kernel "auto" only; q8_gemm_w4a8_ws)."""
    _need(qa, torch.int8, "qa", 2)
    _need(qw4, torch.uint8, "qw4", 2)
    M, K = qa.shape
    N = qw4.shape[0]
    if qw4.shape[1] * 2 != K:
        raise ValueError("qw4 must be [N, K / 2]")
    if out_dtype not in OUT_TYPES:
        raise TypeError("out_dtype must be torch.float32, torch.bfloat16 or torch.int8")
    _need(s_a, torch.float32, "s_a", 1)
    _need(s_w, torch.float32, "s_w", 1)
    if s_a.numel() not in (1, M) or s_w.numel() != N:
        raise ValueError("s_a must have 1 or M entries and s_w N entries")
    ga = Q8_PER_ROW if (s_a.numel() == M and M != 1) else Q8_PER_TENSOR
    if z_a is not None:
        _need(z_a, torch.int32, "z_a", 1)
        if colsum is None:
            raise ValueError("an asymmetric A needs the weight column sums")
        _need(colsum, torch.int32, "colsum", 1)
    if bias is not None:
        _need(bias, torch.float32, "bias", 1)
    if out_dtype == torch.int8 and out_scale is None:
        raise ValueError("int8 output needs out_scale")
    out = torch.empty((M, N), dtype=out_dtype, device=qa.device) if out is None else out
    _need(out, out_dtype, "out", 2)
    if workspace is not None:
        wp, wb = _ws_args(workspace, kernel)
        _check(load().q8_gemm_w4a8_ws(_ptr(qa), _ptr(s_a), _ptr(z_a), ga, _ptr(qw4), _ptr(s_w),
                                      _ptr(colsum if z_a is not None else None), _ptr(bias), M, N, K,
                                      OUT_TYPES[out_dtype], _ptr(out), ctypes.c_float(out_scale or 0.0), wp, wb,
                                      _stream(stream)), "q8_gemm_w4a8_ws")
        return out
    _check(load().q8_gemm_w4a8_ex(_ptr(qa), _ptr(s_a), _ptr(z_a), ga, _ptr(qw4), _ptr(s_w),
                                  _ptr(colsum if z_a is not None else None), _ptr(bias), M, N, K,
                                  OUT_TYPES[out_dtype], _ptr(out), ctypes.c_float(out_scale or 0.0),
                                  KERNELS[kernel], _stream(stream)), "q8_gemm_w4a8")
    return out


def q8_gemm_w4a8_s32(qa, qw4, out=None, kernel: str = "auto", stream=None):
    """Raw INT32 accumulators of int8 qa x packed int4 qw4 (diagnostic export)."""
    _need(qa, torch.int8, "qa", 2)
    _need(qw4, torch.uint8, "qw4", 2)
    M, K = qa.shape
    N = qw4.shape[0]
    out = torch.empty((M, N), dtype=torch.int32, device=qa.device) if out is None else out
    _need(out, torch.int32, "out", 2)
    _check(load().q8_gemm_w4a8_s32_ex(_ptr(qa), _ptr(qw4), M, N, K, _ptr(out), KERNELS[kernel], _stream(stream)),
           "q8_gemm_w4a8_s32")
    return out


def q8_gemm_s32(qa, qw, out=None, kernel: str = "auto", stream=None):
    """Raw INT32 accumulators acc[M, N] = qa . qw^T (diagnostic export of the integer GEMM)."""
    _need(qa, torch.int8, "qa", 2)
    _need(qw, torch.int8, "qw", 2)
    M, K = qa.shape
    N = qw.shape[0]
    out = torch.empty((M, N), dtype=torch.int32, device=qa.device) if out is None else out
    _need(out, torch.int32, "out", 2)
    _check(load().q8_gemm_s32_ex(_ptr(qa), _ptr(qw), M, N, K, _ptr(out), KERNELS[kernel], _stream(stream)),
           "q8_gemm_s32")
    return out


def q8_linear(a, qw, s_w, colsum=None, per_row: bool = True, symmetric: bool = True, kernel: str = "auto",
              qa=None, s_a=None, z_a=None, y=None, workspace=None, stream=None):
    """Whole W8A8 layer on fp32 activations: dynamic quantization of a, then the GEMM + epilogue
    (one C call, q8_linear, for kernel="auto"; an explicit kernel runs the two calls). workspace:
    an optional device tensor of at least q8_gemm_workspace(M, N, K) bytes (q8_linear_ws: the
    quantizer also writes the codes as fp16 values there for the CTA-pair kernel). Returns y."""
    if kernel != "auto":
        qa, s_a, z_a = q8_quantize_act(a, per_row=per_row, symmetric=symmetric, qa=qa, s_a=s_a, z_a=z_a,
                                       stream=stream)
        return q8_gemm_dequant(qa, s_a, z_a, qw, s_w, colsum, kernel=kernel, y=y, stream=stream)
    _need(a, torch.float32, "a", 2)
    _need(qw, torch.int8, "qw", 2)
    _need(s_w, torch.float32, "s_w", 1)
    M, K = a.shape
    N = qw.shape[0]
    if qw.shape[1] != K:
        raise ValueError("qw must be [N, K] with the K of a")
    n = M if per_row else 1
    qa = torch.empty((M, K), dtype=torch.int8, device=a.device) if qa is None else qa
    s_a = torch.empty(n, dtype=torch.float32, device=a.device) if s_a is None else s_a
    if symmetric:
        z_a = None
    elif z_a is None:
        z_a = torch.empty(n, dtype=torch.int32, device=a.device)
    if not symmetric and colsum is None:
        raise ValueError("asymmetric activations need colsum")
    y = torch.empty((M, N), dtype=torch.float32, device=a.device) if y is None else y
    _need(y, torch.float32, "y", 2)
    gw = Q8_PER_ROW if (s_w.numel() == N and N != 1) else Q8_PER_TENSOR
    if workspace is not None:
        wp, wb = _ws_args(workspace, kernel)
        _check(load().q8_linear_ws(_ptr(a), M, K, Q8_PER_ROW if per_row else Q8_PER_TENSOR,
                                   Q8_SYMMETRIC if symmetric else Q8_ASYMMETRIC, _ptr(qa), _ptr(s_a), _ptr(z_a),
                                   _ptr(qw), _ptr(s_w), gw, _ptr(colsum if not symmetric else None), N, _ptr(y), wp,
                                   wb, _stream(stream)), "q8_linear_ws")
        return y
    _check(load().q8_linear(_ptr(a), M, K, Q8_PER_ROW if per_row else Q8_PER_TENSOR,
                            Q8_SYMMETRIC if symmetric else Q8_ASYMMETRIC, _ptr(qa), _ptr(s_a), _ptr(z_a), _ptr(qw),
                            _ptr(s_w), gw, _ptr(colsum if not symmetric else None), N, _ptr(y), _stream(stream)),
           "q8_linear")
    return y


def q8_linear_host_workspace(M: int, N: int, K: int, chunk_rows: int = 0) -> int:
    """Device workspace bytes that q8_linear_host needs."""
    return int(load().q8_linear_host_workspace(M, N, K, chunk_rows))


def q8_linear_host(a_host, qw, s_w, colsum=None, y_host=None, symmetric: bool = True, chunk_rows: int = 0,
                   workspace=None, stream=None):
    """Whole layer on host buffers: a_host fp32 [M, K] (CPU, pinned for overlap) -> y_host fp32 [M, N] (CPU),
    per-token quantization on the device. The result is in y_host once `stream` (default: the current
    stream) has completed."""
    if a_host.device.type != "cpu" or a_host.dtype != torch.float32 or a_host.dim() != 2 or not a_host.is_contiguous():
        raise ValueError("a_host must be a contiguous fp32 [M, K] CPU tensor")
    _need(qw, torch.int8, "qw", 2)
    M, K = a_host.shape
    N = qw.shape[0]
    if qw.shape[1] != K:
        raise ValueError("qw must be [N, K]")
    _need(s_w, torch.float32, "s_w", 1)
    gw = Q8_PER_ROW if (s_w.numel() == N and N != 1) else Q8_PER_TENSOR
    if y_host is None:
        y_host = torch.empty((M, N), dtype=torch.float32, pin_memory=True)
    if y_host.device.type != "cpu" or y_host.dtype != torch.float32 or tuple(y_host.shape) != (M, N) \
            or not y_host.is_contiguous():
        raise ValueError("y_host must be a contiguous fp32 [M, N] CPU tensor")
    need = q8_linear_host_workspace(M, N, K, chunk_rows)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=qw.device)
    _check(load().q8_linear_host(_ptr(a_host), M, K, Q8_SYMMETRIC if symmetric else Q8_ASYMMETRIC, _ptr(qw),
                                 _ptr(s_w), gw, _ptr(colsum), N, _ptr(y_host), chunk_rows, _ptr(workspace),
                                 workspace.numel(), _stream(stream)), "q8_linear_host")
    return y_host


def q8_gemm_pick(M: int, N: int, K: int) -> str:
    return KERNEL_NAMES[load().q8_gemm_pick(M, N, K)]


def q8_launch_count() -> int:
    return int(load().q8_launch_count())


def q8_selftest_wait_timeout(qa, qw, kernel: str = "decode", wait_cycles: int = 1 << 24, stream=None):
    """Self-test of the bounded device waits: runs `kernel` ("decode" or "tcgen05") with its loads
    withheld so that its first wait runs out after wait_cycles; read the result with q8_device_error()."""
    _need(qa, torch.int8, "qa", 2)
    _need(qw, torch.int8, "qw", 2)
    M, K = qa.shape
    N = qw.shape[0]
    acc = torch.zeros((M, N), dtype=torch.int32, device=qa.device)
    _check(load().q8_selftest_wait_timeout(KERNELS[kernel], _ptr(qa), _ptr(qw), M, N, K, _ptr(acc), wait_cycles,
                                           _stream(stream)), "q8_selftest_wait_timeout")
    return acc


def q8_device_error() -> int:
    """Device error word of the tensor-core kernel (0 = every bounded wait completed); resets it."""
    code = ctypes.c_uint32(0)
    st = load().q8_device_error(ctypes.byref(code))
    if st not in (Q8_OK, Q8_ERR_TIMEOUT):
        _check(st, "q8_device_error")
    return int(code.value)


def q8_quantize_weight_mx(w: torch.Tensor, group: int = 32, qw=None, sf=None, stream=None):
    """Block-scaled int8 codes of fp32 W[N, K]: (qw int8 [N, K], sf [ceil(K / group / 4), N] E8M0 scale
    words, held as int32 bit patterns: byte b of word w is group 4w + b)."""
    _need(w, torch.float32, "w", 2)
    N, K = w.shape
    words = (K // group + 3) // 4
    qw = torch.empty((N, K), dtype=torch.int8, device=w.device) if qw is None else qw
    sf = torch.empty((words, N), dtype=torch.int32, device=w.device) if sf is None else sf
    _check(load().q8_quantize_weight_mx(_ptr(w), N, K, group, _ptr(qw), _ptr(sf), _stream(stream)),
           "q8_quantize_weight_mx")
    return qw, sf


def q8_gemm_mx(qa, s_a, qw, sf, group: int = 32, bias=None, out_dtype=torch.float32, out_scale=None, out=None,
               kernel: str = "auto", workspace=None, stream=None):
    """Linear layer with block-scaled int8 weights: y = fl(T * s_a) (+ bias), T = sum_k qa * q * s.
    workspace: as q8_gemm_w4a8 (q8_gemm_mx_ws)."""
    _need(qa, torch.int8, "qa", 2)
    _need(qw, torch.int8, "qw", 2)
    _need(sf, torch.int32, "sf", 2)
    M, K = qa.shape
    N = qw.shape[0]
    if qw.shape[1] != K or sf.shape[1] != N:
        raise ValueError("qw must be [N, K] and sf [words, N]")
    if out_dtype not in OUT_TYPES:
        raise TypeError("out_dtype must be torch.float32, torch.bfloat16 or torch.int8")
    _need(s_a, torch.float32, "s_a", 1)
    if s_a.numel() not in (1, M):
        raise ValueError("s_a must have 1 or M entries")
    ga = Q8_PER_ROW if (s_a.numel() == M and M != 1) else Q8_PER_TENSOR
    if bias is not None:
        _need(bias, torch.float32, "bias", 1)
    if out_dtype == torch.int8 and out_scale is None:
        raise ValueError("int8 output needs out_scale")
    out = torch.empty((M, N), dtype=out_dtype, device=qa.device) if out is None else out
    _need(out, out_dtype, "out", 2)
    if workspace is not None:
        wp, wb = _ws_args(workspace, kernel)
        _check(load().q8_gemm_mx_ws(_ptr(qa), _ptr(s_a), ga, _ptr(qw), _ptr(sf), group, _ptr(bias), M, N, K,
                                    OUT_TYPES[out_dtype], _ptr(out), ctypes.c_float(out_scale or 0.0), wp, wb,
                                    _stream(stream)), "q8_gemm_mx_ws")
        return out
    _check(load().q8_gemm_mx_ex(_ptr(qa), _ptr(s_a), ga, _ptr(qw), _ptr(sf), group, _ptr(bias), M, N, K,
                                OUT_TYPES[out_dtype], _ptr(out), ctypes.c_float(out_scale or 0.0), KERNELS[kernel],
                                _stream(stream)), "q8_gemm_mx")
    return out


# ------------------------------------------------------------- float8 operands, routed experts

FLOAT_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
SCORES = {"softmax": 0, "sigmoid": 1}
FP8_BLOCK = 128
_FP8 = torch.float8_e4m3fn
# A decode step makes many of these calls, so the marshalling is kept short: raw integers for the pointers,
# the stream's handle without a Stream object, each tensor looked at once.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # None in a torch without CUDA


def _cdiv(a: int, b: int) -> int:
    return -(-a // b)


def _float_rows(t: torch.Tensor, name: str):
    """(rows, columns, row pitch, type) of a 2-D CUDA tensor of floats with unit stride along its rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    kind = FLOAT_TYPES.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions")
    rows, cols = t.shape
    pitch, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    if rows <= 1:
        pitch = cols
    elif pitch < cols:
        raise ValueError(f"the rows of {name} overlap")
    return rows, cols, pitch, kind


def _dense(t: torch.Tensor, dtype, shape, device: int, name: str) -> int:
    """The address of a contiguous tensor of this type and shape on the device."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or not t.is_contiguous() or t.get_device() != device:
        _need(t, dtype, name)
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _handle(device: int, stream) -> int:
    """The stream to launch on: of the tensors' device, which has to be the current one."""
    if torch._C._cuda_getDevice() != device:
        raise ValueError(f"the tensors are on cuda:{device}, the current device is cuda:{torch.cuda.current_device()}")
    return _raw_stream(device) if stream is None else stream.cuda_stream


def _out(t, shape, dtype, like: torch.Tensor, device: int, stream, name: str):
    """A result and its address: the caller's tensor, or a new one, allocated on the stream that writes it."""
    if t is not None:
        return t, _dense(t, dtype, shape, device, name)
    if stream is None:
        t = torch.empty(shape, dtype=dtype, device=like.device)
    else:
        with torch.cuda.stream(stream):
            t = torch.empty(shape, dtype=dtype, device=like.device)
    return t, t.data_ptr()


def q8_quantize_fp8(x: torch.Tensor, slots=None, rows: int | None = None, q=None, s=None, stream=None):
    """Float8 codes and scales (one for each row and block of 128) of x[M, K] (fp32, bf16 or fp16; rows may be
    strided). slots int32 [M, k]: row m goes to the rows slots[m] of the result instead (skipped where
    outside), which has `rows` rows (default M * k). Returns (q float8_e4m3fn [rows, K], s fp32 [rows, ceil(K / 128)])."""
    M, K, ldx, kind = _float_rows(x, "x")
    dev = x.get_device()
    top_k, to = 0, None
    if slots is not None:
        if not isinstance(slots, torch.Tensor) or slots.dim() != 2:
            _need(slots, torch.int32, "slots", 2)
        top_k = slots.shape[1]
        to = _dense(slots, torch.int32, (M, top_k), dev, "slots")
        rows = M * top_k if rows is None else rows
    elif rows is not None and rows != M:
        raise ValueError("rows goes with slots")
    else:
        rows = M
    q, pq = _out(q, (rows, K), _FP8, x, dev, stream, "q")
    s, ps = _out(s, (rows, -(-K // FP8_BLOCK)), torch.float32, x, dev, stream, "s")
    status = (_lib or load()).q8_quantize_fp8(x.data_ptr(), kind, M, K, ldx, to, top_k, rows, pq, ps, _handle(dev, stream))
    if status:
        _check(status, "q8_quantize_fp8")
    return q, s


def q8_swiglu_quantize_fp8(h: torch.Tensor, q=None, s=None, stream=None):
    """Codes and scales of silu(h[:, :I]) * h[:, I:], h[M, 2 I] (rows may be strided)."""
    M, cols, ldh, kind = _float_rows(h, "h")
    if cols % 2:
        raise ValueError("h must have an even number of columns")
    I, dev = cols // 2, h.get_device()
    q, pq = _out(q, (M, I), _FP8, h, dev, stream, "q")
    s, ps = _out(s, (M, -(-I // FP8_BLOCK)), torch.float32, h, dev, stream, "s")
    status = (_lib or load()).q8_swiglu_quantize_fp8(h.data_ptr(), kind, M, I, ldh, pq, ps, _handle(dev, stream))
    if status:
        _check(status, "q8_swiglu_quantize_fp8")
    return q, s


def q8_quantize_weight_fp8(w: torch.Tensor, qw=None, sw=None, stream=None):
    """Codes and 128 x 128 block scales of w[N, K] or of the matrices w[E, N, K] (offline)."""
    if not isinstance(w, torch.Tensor) or w.dtype not in FLOAT_TYPES:
        raise TypeError("w must be a float32, bfloat16 or float16 tensor")
    _need(w, w.dtype, "w")
    if w.dim() not in (2, 3):
        raise ValueError("w must be [N, K] or [E, N, K]")
    N, K = w.shape[-2:]
    E = w.shape[0] if w.dim() == 3 else 1
    dev = w.get_device()
    scales = (*w.shape[:-2], _cdiv(N, FP8_BLOCK), _cdiv(K, FP8_BLOCK))
    qw, pq = _out(qw, tuple(w.shape), _FP8, w, dev, stream, "qw")
    sw, ps = _out(sw, scales, torch.float32, w, dev, stream, "sw")
    status = (_lib or load()).q8_quantize_weight_fp8(w.data_ptr(), FLOAT_TYPES[w.dtype], E, N, K, pq, ps, _handle(dev, stream))
    if status:
        _check(status, "q8_quantize_weight_fp8")
    return qw, sw


def _fp8_operands(qa, sa, qw, sw, ndim, out_dtype, out, stream):
    """Addresses and sizes of a product: (device, M, N, K, addresses of qa, sa, qw, sw and out, type, out)."""
    for t, name, dims in ((qa, "qa", 2), (qw, "qw", ndim)):
        if not isinstance(t, torch.Tensor) or t.dtype is not _FP8 or not t.is_cuda or t.dim() != dims or not t.is_contiguous():
            _need(t, _FP8, name, dims)
    M, K = qa.shape
    shape = qw.shape
    N = shape[-2]
    if shape[-1] != K:
        raise ValueError("qa and qw disagree on K")
    kind = FLOAT_TYPES.get(out_dtype)
    if kind is None:
        raise TypeError("out_dtype must be torch.float32, torch.bfloat16 or torch.float16")
    dev, KB, NB = qa.get_device(), -(-K // FP8_BLOCK), -(-N // FP8_BLOCK)
    if qw.get_device() != dev:
        raise ValueError(f"qw is on {qw.device}, not on cuda:{dev}")
    psa = _dense(sa, torch.float32, (M, KB), dev, "sa")
    psw = _dense(sw, torch.float32, (NB, KB) if ndim == 2 else (shape[0], NB, KB), dev, "sw")
    out, py = _out(out, (M, N), out_dtype, qa, dev, stream, "out")
    return dev, M, N, K, qa.data_ptr(), psa, qw.data_ptr(), psw, py, kind, out


def q8_gemm_fp8(qa, sa, qw, sw, out_dtype=torch.bfloat16, out=None, stream=None):
    """y[m, n] = sum over blocks b of sa[m, b] sw[n / 128, b] (qa . qw over block b), as out_dtype [M, N]."""
    dev, M, N, K, pa, psa, pw, psw, py, kind, out = _fp8_operands(qa, sa, qw, sw, 2, out_dtype, out, stream)
    status = (_lib or load()).q8_gemm_fp8(pa, psa, pw, psw, M, N, K, py, kind, _handle(dev, stream))
    if status:
        _check(status, "q8_gemm_fp8")
    return out


def q8_gemm_fp8_grouped(qa, sa, qw, sw, offsets, out_dtype=torch.bfloat16, out=None, stream=None):
    """The product of q8_gemm_fp8 with qw[e] (of qw[E, N, K]) for the rows offsets[e] .. offsets[e + 1] - 1 of each
    expert; offsets int32 [E + 1] stay on the device. Rows of no expert are not written."""
    dev, M, N, K, pa, psa, pw, psw, py, kind, out = _fp8_operands(qa, sa, qw, sw, 3, out_dtype, out, stream)
    E = qw.shape[0]
    status = (_lib or load()).q8_gemm_fp8_grouped(pa, psa, pw, psw,
                                                  _dense(offsets, torch.int32, (E + 1,), dev, "offsets"),
                                                  M, E, N, K, py, kind, _handle(dev, stream))
    if status:
        _check(status, "q8_gemm_fp8_grouped")
    return out


def q8_moe_route(logits: torch.Tensor, top_k: int, score: str = "softmax", bias=None, n_group: int = 1,
                 topk_group: int = 1, renorm: bool = True, scale: float = 1.0, idx=None, weights=None, stream=None):
    """The top_k experts of each token and their weights from logits[T, E] (fp32, bf16 or fp16; rows may be strided):
    (idx int32 [T, top_k], weights fp32 [T, top_k]). score: "softmax" or "sigmoid"; bias fp32 [E] takes part in
    the choice only; with n_group groups only experts of the topk_group best groups are chosen. Masked experts
    (logit -inf or NaN) are not chosen; places that stay empty have idx -1 and weight 0."""
    T, E, ldl, kind = _float_rows(logits, "logits")
    if score not in SCORES:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    if top_k < 1:
        raise ValueError("top_k must be positive")
    dev = logits.get_device()
    pb = None if bias is None else _dense(bias, torch.float32, (E,), dev, "bias")
    idx, pi = _out(idx, (T, top_k), torch.int32, logits, dev, stream, "idx")
    weights, pw = _out(weights, (T, top_k), torch.float32, logits, dev, stream, "weights")
    status = (_lib or load()).q8_moe_route(logits.data_ptr(), kind, T, E, ldl, top_k, SCORES[score], pb, n_group, topk_group,
                               1 if renorm else 0, scale, pi, pw, _handle(dev, stream))
    if status:
        _check(status, "q8_moe_route")
    return idx, weights


def q8_moe_plan(idx: torch.Tensor, n_experts: int, offsets=None, slots=None, stream=None):
    """The choices idx int32 [T, k] sorted by expert (stable): (offsets int32 [n_experts + 1], slots int32 [T, k]),
    the first row of each expert and the row of each choice (-1 where idx is outside [0, n_experts))."""
    if n_experts < 1:
        raise ValueError("n_experts must be positive")
    if not isinstance(idx, torch.Tensor) or idx.dim() != 2 or not idx.is_cuda:
        _need(idx, torch.int32, "idx", 2)
    T, k = idx.shape
    dev = idx.get_device()
    pi = _dense(idx, torch.int32, (T, k), dev, "idx")
    offsets, po = _out(offsets, (n_experts + 1,), torch.int32, idx, dev, stream, "offsets")
    slots, ps = _out(slots, (T, k), torch.int32, idx, dev, stream, "slots")
    status = (_lib or load()).q8_moe_plan(pi, T, k, n_experts, po, ps, _handle(dev, stream))
    if status:
        _check(status, "q8_moe_plan")
    return offsets, slots


def q8_moe_combine(h: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor, out=None, stream=None):
    """y[t] = sum_j weights[t, j] h[slots[t, j]] (fp32 sums), h[rows, N] and y[T, N] of one float type. Slots outside
    [0, rows) add nothing."""
    rows, N, pitch, kind = _float_rows(h, "h")
    if pitch != N:
        raise ValueError("h must be contiguous")
    if not isinstance(slots, torch.Tensor) or slots.dim() != 2:
        _need(slots, torch.int32, "slots", 2)
    T, k = slots.shape
    dev = h.get_device()
    ps = _dense(slots, torch.int32, (T, k), dev, "slots")
    pw = _dense(weights, torch.float32, (T, k), dev, "weights")
    out, py = _out(out, (T, N), h.dtype, h, dev, stream, "out")
    status = (_lib or load()).q8_moe_combine(h.data_ptr(), kind, rows, N, ps, pw, T, k, py, _handle(dev, stream))
    if status:
        _check(status, "q8_moe_combine")
    return out


# --------------------------------------------------------- 4-bit floating point, scales of 16 or 32 K

# The common calls (new results, the current stream) are made by csrc/q8_calls.cpp where it is built, which leaves everything
# else, what is wrong among it, to the functions here by returning None.
FP4_SPAN = 256      # rows of block scales are whole spans of 256 K
_SCALE_TYPES = {16: torch.float8_e4m3fn, 32: torch.float8_e8m0fnu}
_BLOCKS = {v: k for k, v in _SCALE_TYPES.items()}
_VALUE_TYPES = {**FLOAT_TYPES, torch.float8_e4m3fn: 3}


def _fp4_pitch(K: int, block: int) -> int:
    """Block scales of a row, those that fill up its last span among them."""
    return -(-K // FP4_SPAN) * (FP4_SPAN // block)


def _fp4_codes(rows: int, K: int, block: int, q, sf, s, like: torch.Tensor, device: int, stream):
    """Results of a quantizer of `rows` rows: (q, sf, s) and their addresses."""
    kind = _SCALE_TYPES.get(block)
    if kind is None:
        raise ValueError("block must be 16 or 32")
    if K % 32:
        raise ValueError("the number of columns must be a multiple of 32")
    if q is None and sf is None and s is None and stream is None:      # the common call, straight
        on = like.device
        q = torch.empty((rows, K >> 1), dtype=torch.uint8, device=on)
        sf = torch.empty((rows, -(-K // FP4_SPAN) * (FP4_SPAN // block)), dtype=kind, device=on)
        if block == 32:
            return q, sf, None, q.data_ptr(), sf.data_ptr(), None
        s = torch.empty(rows, dtype=torch.float32, device=on)
        return q, sf, s, q.data_ptr(), sf.data_ptr(), s.data_ptr()
    q, pq = _out(q, (rows, K // 2), torch.uint8, like, device, stream, "q")
    sf, psf = _out(sf, (rows, _fp4_pitch(K, block)), kind, like, device, stream, "sf")
    if block == 32:
        if s is not None:
            raise ValueError("s goes with block 16")
        return q, sf, None, pq, psf, None
    s, ps = _out(s, (rows,), torch.float32, like, device, stream, "s")
    return q, sf, s, pq, psf, ps


def q8_quantize_fp4(x: torch.Tensor, block: int = 16, slots=None, rows: int | None = None, q=None, sf=None, s=None, stream=None):
    """4-bit codes of x[M, K] (fp32, bf16 or fp16; rows may be strided; K a multiple of 32). block 16: e4m3 scales of 16 K under an
    fp32 scale a row; block 32: powers of two of 32 K. slots int32 [M, k]: row m goes to the rows slots[m] of the result instead
    (skipped where outside), which has `rows` rows (default M * k). Returns (q uint8 [rows, K / 2], two codes a byte, sf
    [rows, 256 / block * ceil(K / 256)] float8_e4m3fn or float8_e8m0fnu, s fp32 [rows] or None)."""
    if _calls is not None and rows is None and q is None and sf is None and s is None and stream is None:
        got = _calls.quantize_fp4(x, block, slots)
        if got is not None:
            return got
    M, K, ldx, kind = _float_rows(x, "x")
    dev = x.get_device()
    top_k, to = 0, None
    if slots is not None:
        if not isinstance(slots, torch.Tensor) or slots.dim() != 2:
            _need(slots, torch.int32, "slots", 2)
        top_k = slots.shape[1]
        to = _dense(slots, torch.int32, (M, top_k), dev, "slots")
        rows = M * top_k if rows is None else rows
    elif rows is not None and rows != M:
        raise ValueError("rows goes with slots")
    else:
        rows = M
    q, sf, s, pq, psf, ps = _fp4_codes(rows, K, block, q, sf, s, x, dev, stream)
    status = (_lib or load()).q8_quantize_fp4(x.data_ptr(), kind, block, M, K, ldx, to, top_k, rows, pq, psf, ps,
                                              _handle(dev, stream))
    if status:
        _check(status, "q8_quantize_fp4")
    return q, sf, s


def q8_swiglu_quantize_fp4(h: torch.Tensor, block: int = 16, q=None, sf=None, s=None, stream=None):
    """Codes and scales (as q8_quantize_fp4) of silu(h[:, :I]) * h[:, I:], h[M, 2 I] (rows may be strided)."""
    if _calls is not None and q is None and sf is None and s is None and stream is None:
        got = _calls.swiglu_quantize_fp4(h, block)
        if got is not None:
            return got
    M, cols, ldh, kind = _float_rows(h, "h")
    if cols % 2:
        raise ValueError("h must have an even number of columns")
    I, dev = cols // 2, h.get_device()
    q, sf, s, pq, psf, ps = _fp4_codes(M, I, block, q, sf, s, h, dev, stream)
    status = (_lib or load()).q8_swiglu_quantize_fp4(h.data_ptr(), kind, block, M, I, ldh, pq, psf, ps, _handle(dev, stream))
    if status:
        _check(status, "q8_swiglu_quantize_fp4")
    return q, sf, s


def _fp4_tiles(N: int, K: int, block: int):
    """Shape of the block scales of a weight matrix: tiles of 128 rows x 4 scales."""
    return _cdiv(N, 128), _fp4_pitch(K, block) // 4, 32, 4, 4


def q8_quantize_weight_fp4(w: torch.Tensor, block: int = 16, qw=None, sfw=None, sw=None, stream=None):
    """4-bit codes of w[N, K] or of the matrices w[E, N, K] (offline): (qw uint8 [.., N, K / 2], sfw [.., ceil(N / 128),
    64 / block * ceil(K / 256), 32, 4, 4], sw fp32 [.., N] or None). Scale b of row n is at
    sfw[n // 128, b // 4, n % 32, n % 128 // 32, b % 4]."""
    if not isinstance(w, torch.Tensor) or w.dtype not in FLOAT_TYPES:
        raise TypeError("w must be a float32, bfloat16 or float16 tensor")
    _need(w, w.dtype, "w")
    if w.dim() not in (2, 3):
        raise ValueError("w must be [N, K] or [E, N, K]")
    kind = _SCALE_TYPES.get(block)
    if kind is None:
        raise ValueError("block must be 16 or 32")
    N, K = w.shape[-2:]
    if K % 32:
        raise ValueError("the number of columns must be a multiple of 32")
    lead, dev = tuple(w.shape[:-2]), w.get_device()
    E = lead[0] if lead else 1
    qw, pq = _out(qw, (*lead, N, K // 2), torch.uint8, w, dev, stream, "qw")
    sfw, psf = _out(sfw, (*lead, *_fp4_tiles(N, K, block)), kind, w, dev, stream, "sfw")
    ps = None
    if block == 16:
        sw, ps = _out(sw, (*lead, N), torch.float32, w, dev, stream, "sw")
    elif sw is not None:
        raise ValueError("sw goes with block 16")
    status = (_lib or load()).q8_quantize_weight_fp4(w.data_ptr(), FLOAT_TYPES[w.dtype], block, E, N, K, pq, psf, ps,
                                                     _handle(dev, stream))
    if status:
        _check(status, "q8_quantize_weight_fp4")
    return qw, sfw, sw


def q8_dequantize_fp4(q: torch.Tensor, sf=None, s=None, out_dtype=torch.bfloat16, out=None, stream=None):
    """What codes stand for, [.., K]: q (q8_quantize_fp4's [rows, K / 2] or q8_quantize_weight_fp4's) times its block scales sf (of the
    same kind) times its row scales s; without a scale it counts as 1. out_dtype float32, bfloat16 or float16; without scales
    also float8_e4m3fn, which holds every code."""
    if _calls is not None and sf is None and s is None and out is None and stream is None:
        got = _calls.dequantize_fp4(q, out_dtype)
        if got is not None:
            return got
    if not isinstance(q, torch.Tensor) or q.dtype is not torch.uint8 or not q.is_cuda or q.dim() not in (2, 3):
        _need(q, torch.uint8, "q")
        raise ValueError("q must be [rows, K / 2] or [E, N, K / 2]")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    kind = _VALUE_TYPES.get(out_dtype)
    if kind is None:
        raise TypeError("out_dtype must be torch.float32, torch.bfloat16, torch.float16 or torch.float8_e4m3fn")
    if kind == 3 and (sf is not None or s is not None):
        raise ValueError("float8 holds the codes alone, without scales")
    dev = q.get_device()
    if sf is None and s is None:                                       # the codes alone
        shape = (*q.shape[:-1], 2 * q.shape[-1])
        out, py = _out(out, shape, out_dtype, q, dev, stream, "out")
        status = (_lib or load()).q8_dequantize_fp4(q.data_ptr(), None, None, 16, q.numel() // max(1, q.shape[-1]), shape[-1], 0, py,
                                                    kind, _handle(dev, stream))
        if status:
            _check(status, "q8_dequantize_fp4")
        return out
    lead, N, K = tuple(q.shape[:-2]), q.shape[-2], 2 * q.shape[-1]
    rows, block, tile_rows, psf, ps = (lead[0] * N if lead else N), 16, 0, None, None
    if sf is not None:
        block = _BLOCKS.get(sf.dtype) if isinstance(sf, torch.Tensor) else None
        if block is None:
            raise TypeError("sf must be float8_e4m3fn (blocks of 16) or float8_e8m0fnu (blocks of 32)")
        if sf.dim() == 2 and not lead:
            psf = _dense(sf, sf.dtype, (N, _fp4_pitch(K, block)), dev, "sf")
        else:
            psf, tile_rows = _dense(sf, sf.dtype, (*lead, *_fp4_tiles(N, K, block)), dev, "sf"), N
    if s is not None:
        ps = _dense(s, torch.float32, (*lead, N), dev, "s")
    out, py = _out(out, (*lead, N, K), out_dtype, q, dev, stream, "out")
    status = (_lib or load()).q8_dequantize_fp4(q.data_ptr(), psf, ps, block, rows, K, tile_rows, py, kind, _handle(dev, stream))
    if status:
        _check(status, "q8_dequantize_fp4")
    return out


def _fp4_operands(qa, sfa, sa, qw, sfw, sw, ndim, out_dtype, out, stream):
    """Addresses and sizes of a product: (device, M, N, K, block, addresses of qa, sfa, sa, qw, sfw, sw and out, type, out)."""
    u8 = torch.uint8
    if not isinstance(qa, torch.Tensor) or qa.dtype is not u8 or not qa.is_cuda or qa.dim() != 2 or not qa.is_contiguous():
        _need(qa, u8, "qa", 2)
    if not isinstance(qw, torch.Tensor) or qw.dtype is not u8 or not qw.is_cuda or qw.dim() != ndim or not qw.is_contiguous():
        _need(qw, u8, "qw", ndim)
    scales = sfa.dtype if isinstance(sfa, torch.Tensor) else None
    block = _BLOCKS.get(scales)
    if block is None:
        raise TypeError("sfa must be float8_e4m3fn (blocks of 16) or float8_e8m0fnu (blocks of 32)")
    M, half = qa.shape
    shape = qw.shape
    N, K = shape[-2], 2 * half
    if shape[-1] != half:
        raise ValueError("qa and qw disagree on K")
    kind = FLOAT_TYPES.get(out_dtype)
    if kind is None:
        raise TypeError("out_dtype must be torch.float32, torch.bfloat16 or torch.float16")
    dev = qa.get_device()
    if qw.get_device() != dev:
        raise ValueError(f"qw is on {qw.device}, not on cuda:{dev}")
    pitch = -(-K // FP4_SPAN) * (FP4_SPAN // block)
    psfa = _dense(sfa, scales, (M, pitch), dev, "sfa")
    if ndim == 2:
        psfw = _dense(sfw, scales, (-(-N // 128), pitch >> 2, 32, 4, 4), dev, "sfw")
        psw = None if sw is None else _dense(sw, torch.float32, (N,), dev, "sw")
    else:
        psfw = _dense(sfw, scales, (shape[0], -(-N // 128), pitch >> 2, 32, 4, 4), dev, "sfw")
        psw = None if sw is None else _dense(sw, torch.float32, (shape[0], N), dev, "sw")
    psa = None if sa is None else _dense(sa, torch.float32, (M,), dev, "sa")
    out, py = _out(out, (M, N), out_dtype, qa, dev, stream, "out")
    return dev, M, N, K, block, qa.data_ptr(), psfa, psa, qw.data_ptr(), psfw, psw, py, kind, out


def q8_gemm_fp4(qa, sfa, sa, qw, sfw, sw, out_dtype=torch.bfloat16, out=None, stream=None):
    """y[m, n] = sa[m] sw[n] sum over blocks b of sfa[m, b] sfw[n, b] (qa . qw over block b), as out_dtype [M, N]. The operands are
    those of q8_quantize_fp4 and q8_quantize_weight_fp4, with the same block; sa or sw None stands for ones."""
    if _calls is not None and out is None and stream is None:
        got = _calls.gemm_fp4(qa, sfa, sa, qw, sfw, sw, None, out_dtype)
        if got is not None:
            return got
    dev, M, N, K, block, pa, psfa, psa, pw, psfw, psw, py, kind, out = _fp4_operands(qa, sfa, sa, qw, sfw, sw, 2, out_dtype, out,
                                                                                     stream)
    status = (_lib or load()).q8_gemm_fp4(pa, psfa, psa, pw, psfw, psw, block, M, N, K, py, kind, _handle(dev, stream))
    if status:
        _check(status, "q8_gemm_fp4")
    return out


def q8_gemm_fp4_grouped(qa, sfa, sa, qw, sfw, sw, offsets, out_dtype=torch.bfloat16, out=None, stream=None):
    """The product of q8_gemm_fp4 with qw[e], sfw[e], sw[e] (of qw[E, N, K / 2]) for the rows offsets[e] .. offsets[e + 1] - 1 of each
    expert; offsets int32 [E + 1] stay on the device. Rows of no expert are not written."""
    if _calls is not None and offsets is not None and out is None and stream is None:
        got = _calls.gemm_fp4(qa, sfa, sa, qw, sfw, sw, offsets, out_dtype)
        if got is not None:
            return got
    dev, M, N, K, block, pa, psfa, psa, pw, psfw, psw, py, kind, out = _fp4_operands(qa, sfa, sa, qw, sfw, sw, 3, out_dtype, out,
                                                                                     stream)
    E = qw.shape[0]
    status = (_lib or load()).q8_gemm_fp4_grouped(pa, psfa, psa, pw, psfw, psw,
                                                  _dense(offsets, torch.int32, (E + 1,), dev, "offsets"), block, M, E, N, K, py,
                                                  kind, _handle(dev, stream))
    if status:
        _check(status, "q8_gemm_fp4_grouped")
    return out
