"""AWQ W4A16 g128 for NVIDIA B200 — Python binding of ``libawq_w4a16.so``.

The binding only marshals arguments: it checks tensor dtypes, shapes and
devices, allocates outputs with PyTorch when the caller gives none, and
passes raw device pointers plus the current CUDA stream to the C ABI declared
in ``include/awq_w4a16.h``. Every step of the path runs in the library's
CUDA kernels; if the library is missing, every call raises.

Functions (same names as the C ABI):

* ``awq_activation_scale(x, alpha)``  -> (s[K] fp32, x'[M,K] fp16)
* ``awq_scale_activations(x, s)`` -> x'[M,K] fp16 with a stored s
* ``awq_quantize_g128(W, fold_scale)`` -> (qweight int32, scales fp16, zeros uint8)
* ``awq_w4a16_gemv(x, qweight, scales, zeros, N)`` -> y[M,N] fp16 (M <= 32)
* ``awq_w4a16_gemm(x, qweight, scales, zeros, N)`` -> y[M,N] fp16
* ``awq_w4a16_linear(...)``: gemv for M <= 32, gemm otherwise
* ``awq_w4a16_linear_qkv(x, qweight, scales, zeros, Nq, Nkv)`` -> (q, k, v): fused q/k/v split
* ``awq_w4a16_linear_silu_mul(x, qweight, scales, zeros, I)`` -> h = SiLU(gate) * up
* ``awq_search_alpha(x, W, alphas)`` -> (err[n] float64, best index): the AWQ scale search
* ``awq_quantize_tokens(x, s)`` -> (xq int8, sx fp32); ``awq_quantize_channels(W, fold_scale)`` -> (wq, sw)
* ``awq_w8a8_linear(xq, sx, wq, sw)`` -> y[M,N] fp16: the product in 8-bit integers;
  ``awq_w8a8_forward(x, wq, sw, s)`` with the tokens' quantization; class ``AWQInt8Linear``
* ``awq_residual_norm(y, residual, weight, ...)`` -> (h, x'): residual update, RMS norms, activation scaling
* ``awq_moe_w4a16(x, router, gate_up, down, I, top_k)`` -> y[T,K]: a mixture-of-experts layer for a few
  tokens, experts in packed weights; class ``AWQMoE``
* ``awq_poll_device_status()``, test hooks ``awq_debug_set_wait_budget_ns(ns)``,
  ``awq_debug_drop_first_copy(enable)``, ``awq_debug_set_gemm_split(ks)``
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libawq_w4a16.so")

AWQ_OK = 0
AWQ_ERR_INVALID_ARG = 1
AWQ_ERR_UNSUPPORTED = 2
AWQ_ERR_MISALIGNED = 3
AWQ_ERR_CUDA = 4
AWQ_ERR_TIMEOUT = 5
AWQ_ERR_BOUNDS = 6    # debug builds only

GROUP_SIZE = 128
BITS = 4

_lib = None


class AWQError(RuntimeError):
    """A C-ABI call returned a status other than AWQ_OK."""

    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {msg}")
        self.status = status


_VP = ctypes.c_void_p
_I = ctypes.c_int
_SIGS = {
    "awq_layout_version": ([], ctypes.c_int),
    "awq_status_string": ([_I], ctypes.c_char_p),
    "awq_check_config": ([_I, _I, _I], _I),
    "awq_qweight_bytes": ([_I, _I], ctypes.c_size_t),
    "awq_scales_bytes": ([_I, _I], ctypes.c_size_t),
    "awq_zeros_bytes": ([_I, _I], ctypes.c_size_t),
    "awq_activation_scale": ([_VP, _I, _I, ctypes.c_float, _VP, _VP, _VP], _I),
    "awq_scale_activations": ([_VP, _VP, _I, _I, _VP, _VP], _I),
    "awq_quantize_g128": ([_VP, _VP, _I, _I, _VP, _VP, _VP, _VP], _I),
    "awq_quantize": ([_VP, _VP, _I, _I, _I, _I, _I, _VP, _VP, _VP, _VP], _I),
    "awq_w4a16_gemv": ([_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _VP], _I),
    "awq_w4a16_gemm": ([_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _VP], _I),
    "awq_w4a16_linear": ([_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _VP], _I),
    "awq_poll_device_status": ([_VP], _I),
    "awq_search_workspace_bytes": ([_I, _I, _I], ctypes.c_size_t),
    "awq_w4a16_linear_qkv": ([_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _VP], _I),
    "awq_w4a16_linear_silu_mul": ([_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _VP], _I),
    "awq_search_alpha": ([_VP, _VP, _I, _I, _I, _VP, _I, _VP, _VP, _VP, ctypes.c_size_t, _VP], _I),
    "awq_search_alpha_noalloc": ([_VP, _VP, _I, _I, _I, _VP, _I, _VP, _VP, _VP], _I),
    "awq_quantize_tokens": ([_VP, _VP, _I, _I, _VP, _VP, _VP], _I),
    "awq_quantize_channels": ([_VP, _VP, _I, _I, _VP, _VP, _VP], _I),
    "awq_w8a8_linear": ([_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _VP], _I),
    "awq_w8a8_workspace_bytes": ([_I, _I], ctypes.c_size_t),
    "awq_w8a8_forward": ([_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _VP, ctypes.c_size_t, _VP], _I),
    "awq_residual_norm": ([_VP, _VP, _VP, _I, _VP, _VP, _VP, ctypes.c_float, ctypes.c_float, _I, _I, _VP, _VP, _VP], _I),
    "awq_moe_workspace_bytes": ([_I, _I, _I, _I, _I], ctypes.c_size_t),
    "awq_moe_w4a16": ([_VP] * 9 + [_I] * 6 + [_VP, _VP, ctypes.c_size_t, _VP], _I),
    "awq_debug_set_wait_budget_ns": ([ctypes.c_ulonglong], _I),
    "awq_debug_drop_first_copy": ([_I], _I),
    "awq_debug_set_gemm_split": ([_I], _I),
    "awq_gemm_plan": ([_I, _I, _I, _I, _I, ctypes.POINTER(_I), ctypes.POINTER(_I), ctypes.POINTER(ctypes.c_longlong)],
                      _I),
}


def library_path() -> str:
    return LIB_PATH


def load_library(path: Optional[str] = None):
    """Loads libawq_w4a16.so (built in-tree by ``build.py``). Raises if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"{p} is missing: build it with `python -m weight_only_quantization_w4a16_b200.build` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(p)
    for name, (args, res) in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path is None:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().awq_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != AWQ_OK:
        raise AWQError(fn, status, status_string(status))


LAYOUT_VERSION = 2   # the packed-weight layout this binding's size checks assume


def layout_version() -> int:
    return int(load_library().awq_layout_version())


def check_config(bits: int, group_size: int, zero_point: bool) -> bool:
    return load_library().awq_check_config(int(bits), int(group_size), int(bool(zero_point))) == AWQ_OK


def packed_nbytes(N: int, K: int) -> Tuple[int, int, int]:
    lib = load_library()
    return (int(lib.awq_qweight_bytes(N, K)), int(lib.awq_scales_bytes(N, K)), int(lib.awq_zeros_bytes(N, K)))


# ---------------------------------------------------------------------------- torch marshalling
# The calls are a few microseconds of GPU work at their smallest, so the checks below are written to
# cost little when they pass: one expression per tensor, the message worked out only on a failure.
_torch_mod = None


def _torch():
    global _torch_mod
    if _torch_mod is None:
        import torch
        _torch_mod = torch
    return _torch_mod


_raw_stream = None     # current stream handle of a device, without building a Stream object where torch allows it


def _stream_ptr(device=None):
    """The current stream's handle on `device`, the current one where the caller does not know it already."""
    global _raw_stream
    if _raw_stream is None:
        torch = _torch()
        torch.cuda.init()
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
    return _raw_stream(_torch().cuda.current_device() if device is None else device)


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _fits(t, dtype, dims: int, numel: int, device: int) -> bool:
    """Whether t is a contiguous tensor of this type and size on the given (current) device: what the
    validators check, without their messages. The calls that are made once per token ask this first."""
    return (type(t) is _torch_mod.Tensor and t.dtype is dtype and t.dim() == dims and t.numel() == numel and
            t.get_device() == device and t.is_contiguous())


def _need(t, dtype, name, dims=None, require_cuda=True):
    torch = _torch_mod or _torch()
    if (type(t) is torch.Tensor and t.dtype is dtype and t.is_contiguous() and (dims is None or t.dim() == dims) and
            (not require_cuda or (t.is_cuda and t.get_device() == torch.cuda.current_device()))):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if require_cuda:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.device.index != torch.cuda.current_device():
            raise ValueError(f"{name} is on {t.device}, but the current CUDA device is "
                             f"cuda:{torch.cuda.current_device()} (the library runs on the current device)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions")


def _packed_sizes_host(N: int, K: int) -> Tuple[int, int, int]:
    """Byte sizes of packed layout v2 computed here (used before a library call, so that a caller's
    buffers are checked against the same figures the library states)."""
    if N < 1 or K < GROUP_SIZE or K % GROUP_SIZE:
        return 0, 0, 0
    tiles, pairs = -(-N // 16), -(-(K // GROUP_SIZE) // 2)
    return tiles * pairs * 2048, tiles * pairs * 64, tiles * pairs * 16


def _check_packed(qweight, scales, zeros, N: int, K: int, require_cuda=True):
    torch = _torch()
    _need(qweight, torch.int32, "qweight", require_cuda=require_cuda)
    _need(scales, torch.float16, "scales", require_cuda=require_cuda)
    _need(zeros, torch.uint8, "zeros", require_cuda=require_cuda)
    qb, sb, zb = _packed_sizes_host(N, K)
    if qb == 0:
        raise ValueError("N >= 1 and K a positive multiple of 128 are required")
    if qweight.numel() * 4 < qb or scales.numel() * 2 < sb or zeros.numel() < zb:
        raise ValueError(f"packed weight tensors are too small for N={N}, K={K}: need {qb}, {sb}, {zb} bytes")


def _check_vec(v, K: int, name: str, require_cuda=True):
    torch = _torch()
    _need(v, torch.float32, name, 1, require_cuda=require_cuda)
    if v.numel() != K:
        raise ValueError(f"{name} must have K={K} elements, got {v.numel()}")


def validate_activation_scale(x, s_out, x_scaled, require_cuda=True):
    torch = _torch()
    _need(x, torch.float16, "x", 2, require_cuda=require_cuda)
    M, K = x.shape
    _check_vec(s_out, K, "s_out", require_cuda)
    if x_scaled is not None:
        _need(x_scaled, torch.float16, "x_scaled", 2, require_cuda=require_cuda)
        if tuple(x_scaled.shape) != (M, K):
            raise ValueError(f"x_scaled must have shape {(M, K)}, got {tuple(x_scaled.shape)}")


def validate_scale_activations(x, s, x_scaled, require_cuda=True):
    torch = _torch()
    _need(x, torch.float16, "x", 2, require_cuda=require_cuda)
    M, K = x.shape
    _check_vec(s, K, "s", require_cuda)
    _need(x_scaled, torch.float16, "x_scaled", 2, require_cuda=require_cuda)
    if tuple(x_scaled.shape) != (M, K):
        raise ValueError(f"x_scaled must have shape {(M, K)}, got {tuple(x_scaled.shape)}")


def validate_quantize(W, fold_scale, out, require_cuda=True):
    torch = _torch()
    _need(W, torch.float16, "W", 2, require_cuda=require_cuda)
    N, K = W.shape
    if fold_scale is not None:
        _check_vec(fold_scale, K, "fold_scale", require_cuda)
    _check_packed(*out, N, K, require_cuda=require_cuda)


def validate_linear(x, qweight, scales, zeros, N: int, y, require_cuda=True):
    torch = _torch()
    _need(x, torch.float16, "x", 2, require_cuda=require_cuda)
    M, K = x.shape
    _check_packed(qweight, scales, zeros, N, K, require_cuda=require_cuda)
    _need(y, torch.float16, "y", 2, require_cuda=require_cuda)
    if tuple(y.shape) != (M, N):
        raise ValueError(f"y must have shape {(M, N)}, got {tuple(y.shape)}")


def awq_activation_scale(x, alpha: float = 0.5, s_out=None, x_scaled=None, want_scaled: bool = True):
    """a1: s[K] = max(mean_m |x[m,k]|, 1e-8)^alpha and x' = fp16(x / s)."""
    torch = _torch()
    _need(x, torch.float16, "x", 2)
    M, K = x.shape
    if s_out is None:
        s_out = torch.empty(K, dtype=torch.float32, device=x.device)
    if want_scaled and x_scaled is None:
        x_scaled = torch.empty_like(x)
    validate_activation_scale(x, s_out, x_scaled)
    st = load_library().awq_activation_scale(_ptr(x), M, K, float(alpha), _ptr(s_out), _ptr(x_scaled),
                                             _stream_ptr())
    _check("awq_activation_scale", st)
    return s_out, x_scaled


def alloc_packed(N: int, K: int, device="cuda"):
    """Output tensors for awq_quantize_g128: qweight (int32 words), scales (fp16), zeros (uint8)."""
    torch = _torch()
    qb, sb, zb = packed_nbytes(N, K)
    if qb == 0:
        raise ValueError("N >= 1 and K a positive multiple of 128 are required")
    return (torch.empty(qb // 4, dtype=torch.int32, device=device),
            torch.empty(sb // 2, dtype=torch.float16, device=device),
            torch.empty(zb, dtype=torch.uint8, device=device))


def awq_quantize_g128(W, fold_scale=None, out=None):
    """a2: fold s into W[N,K] and quantize to packed layout v2. Returns (qweight, scales, zeros)."""
    torch = _torch()
    _need(W, torch.float16, "W", 2)
    N, K = W.shape
    out = out if out is not None else alloc_packed(N, K, W.device)
    validate_quantize(W, fold_scale, out)
    qweight, scales, zeros = out
    st = load_library().awq_quantize_g128(_ptr(W), _ptr(fold_scale), N, K, _ptr(qweight), _ptr(scales),
                                          _ptr(zeros), _stream_ptr())
    _check("awq_quantize_g128", st)
    return qweight, scales, zeros


def awq_quantize(W, fold_scale=None, bits: int = 4, group_size: int = 128, zero_point: bool = True, out=None):
    """a2 variants: INT4 or INT3 codes, asymmetric (zero_point) or symmetric, group size 128, in
    packed layout v2. Returns (qweight, scales, zeros)."""
    torch = _torch()
    _need(W, torch.float16, "W", 2)
    N, K = W.shape
    out = out if out is not None else alloc_packed(N, K, W.device)
    validate_quantize(W, fold_scale, out)
    qweight, scales, zeros = out
    st = load_library().awq_quantize(_ptr(W), _ptr(fold_scale), N, K, int(bits), int(group_size), int(bool(zero_point)),
                                     _ptr(qweight), _ptr(scales), _ptr(zeros), _stream_ptr())
    _check("awq_quantize", st)
    return qweight, scales, zeros


def _linear(fn_name: str, x, qweight, scales, zeros, N: int, y=None):
    torch = _torch()
    _need(x, torch.float16, "x", 2)
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=x.device)
    validate_linear(x, qweight, scales, zeros, N, y)
    st = getattr(load_library(), fn_name)(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(y), M, N, K,
                                          _stream_ptr())
    _check(fn_name, st)
    return y


def awq_w4a16_gemv(x, qweight, scales, zeros, N: int, y=None):
    """a3: y[M,N] = x' . dequant^T for M <= 32 (decode)."""
    return _linear("awq_w4a16_gemv", x, qweight, scales, zeros, N, y)


def awq_w4a16_gemm(x, qweight, scales, zeros, N: int, y=None):
    """a4: y[M,N] = x' . dequant^T on tcgen05 tensor cores (prefill)."""
    return _linear("awq_w4a16_gemm", x, qweight, scales, zeros, N, y)


def awq_w4a16_linear(x, qweight, scales, zeros, N: int, y=None):
    """The decode kernel for small M, the prefill kernel otherwise (the library picks)."""
    return _linear("awq_w4a16_linear", x, qweight, scales, zeros, N, y)


def awq_w4a16_linear_qkv(x, qweight, scales, zeros, Nq: int, Nkv: int, out=None):
    """Fused q/k/v layer (weight rows: Nq query, Nkv key, Nkv value); returns (q, k, v)."""
    torch = _torch()
    _need(x, torch.float16, "x", 2)
    M, K = x.shape
    N = Nq + 2 * Nkv
    if out is None:
        out = tuple(torch.empty((M, n), dtype=torch.float16, device=x.device) for n in (Nq, Nkv, Nkv))
    _check_packed(qweight, scales, zeros, N, K)
    for t, n, name in zip(out, (Nq, Nkv, Nkv), ("q", "k", "v")):
        _need(t, torch.float16, name, 2)
        if tuple(t.shape) != (M, n):
            raise ValueError(f"{name} must have shape {(M, n)}")
    st = load_library().awq_w4a16_linear_qkv(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(zeros), *[_ptr(t) for t in out],
                                             M, Nq, Nkv, K, _stream_ptr())
    _check("awq_w4a16_linear_qkv", st)
    return out


def awq_w4a16_linear_silu_mul(x, qweight, scales, zeros, I: int, h=None):
    """Fused gate+up layer (weight rows: I gate, then I up; I % 16 == 0): h = SiLU(gate) * up."""
    torch = _torch()
    _need(x, torch.float16, "x", 2)
    M, K = x.shape
    if I < 16 or I % 16:
        raise ValueError("I must be a positive multiple of 16")
    if h is None:
        h = torch.empty((M, I), dtype=torch.float16, device=x.device)
    _check_packed(qweight, scales, zeros, 2 * I, K)
    _need(h, torch.float16, "h", 2)
    if tuple(h.shape) != (M, I):
        raise ValueError(f"h must have shape {(M, I)}")
    st = load_library().awq_w4a16_linear_silu_mul(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(h), M, I,
                                                  K, _stream_ptr())
    _check("awq_w4a16_linear_silu_mul", st)
    return h


def awq_search_alpha(x, W, alphas=None, workspace=None):
    """AWQ scale search: the squared output error of the whole path for every candidate exponent.

    ``alphas`` defaults to an even grid of 20 points over [0, 1). Returns (err, best, alphas) with
    err a float64 CUDA tensor and best a one-element int32 CUDA tensor (no host synchronization).
    """
    torch = _torch()
    _need(x, torch.float16, "x", 2)
    _need(W, torch.float16, "W", 2)
    M, K = x.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError(f"W must have K={K} columns")
    if alphas is None:
        alphas = [i / 20.0 for i in range(20)]
    a = (ctypes.c_float * len(alphas))(*[float(v) for v in alphas])
    lib = load_library()
    need = int(lib.awq_search_workspace_bytes(M, N, K))
    if need == 0:
        raise ValueError("shape out of range for the search")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    _need(workspace, torch.uint8, "workspace", 1)
    if workspace.numel() < need:
        raise ValueError(f"workspace must hold {need} bytes")
    err = torch.empty(len(alphas), dtype=torch.float64, device=x.device)
    best = torch.empty(1, dtype=torch.int32, device=x.device)
    st = lib.awq_search_alpha(_ptr(x), _ptr(W), M, N, K, ctypes.cast(a, _VP), len(alphas), _ptr(err), _ptr(best),
                              _ptr(workspace), workspace.numel(), _stream_ptr())
    _check("awq_search_alpha", st)
    return err, best, list(alphas)


SEARCH_NOALLOC_SCRATCH_BYTES = 64 << 20   # the fixed scratch of awq_search_alpha_noalloc


def awq_search_alpha_noalloc(x, W, alphas=None):
    """The scale search on the library's fixed device scratch (no workspace argument).

    For callers that cannot allocate device memory themselves; results equal awq_search_alpha's.
    Shapes whose workspace would exceed SEARCH_NOALLOC_SCRATCH_BYTES raise ValueError. Only the
    outputs err and best are allocated here, by the caller's framework.
    """
    torch = _torch()
    _need(x, torch.float16, "x", 2)
    _need(W, torch.float16, "W", 2)
    M, K = x.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError(f"W must have K={K} columns")
    if alphas is None:
        alphas = [i / 20.0 for i in range(20)]
    a = (ctypes.c_float * len(alphas))(*[float(v) for v in alphas])
    lib = load_library()
    need = int(lib.awq_search_workspace_bytes(M, N, K))
    if need == 0 or need > SEARCH_NOALLOC_SCRATCH_BYTES:
        raise ValueError(f"shape out of range for the search without workspace ({need} bytes needed)")
    err = torch.empty(len(alphas), dtype=torch.float64, device=x.device)
    best = torch.empty(1, dtype=torch.int32, device=x.device)
    st = lib.awq_search_alpha_noalloc(_ptr(x), _ptr(W), M, N, K, ctypes.cast(a, _VP), len(alphas), _ptr(err),
                                      _ptr(best), _stream_ptr())
    _check("awq_search_alpha_noalloc", st)
    return err, best, list(alphas)


def awq_poll_device_status() -> int:
    """Synchronizes the current stream and returns (and clears) the device status code."""
    return int(load_library().awq_poll_device_status(_stream_ptr()))


def awq_debug_set_wait_budget_ns(ns: int) -> None:
    _check("awq_debug_set_wait_budget_ns", load_library().awq_debug_set_wait_budget_ns(int(ns)))


def awq_debug_drop_first_copy(enable: bool) -> None:
    _check("awq_debug_drop_first_copy", load_library().awq_debug_drop_first_copy(int(bool(enable))))


def awq_gemm_plan(M: int, N: int, K: int, epilogue: int = 0, num_sms: Optional[int] = None) -> Tuple[int, int, int]:
    """(token tile, K split, split tiles) that the prefill kernel takes for this shape (host-only).
    epilogue: 0 plain, 1 q/k/v split, 2 gate/up SiLU*up; num_sms defaults to the current device's."""
    if num_sms is None:
        import torch
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    bt, ks, nsplit = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_longlong(0)
    _check("awq_gemm_plan", load_library().awq_gemm_plan(int(M), int(N), int(K), int(epilogue), int(num_sms),
                                                          ctypes.byref(bt), ctypes.byref(ks), ctypes.byref(nsplit)))
    return bt.value, ks.value, nsplit.value


def awq_debug_set_gemm_split(ks: int) -> None:
    """Prefill K split: 0 chooses per launch, 1 never splits, 2 splits every tile across a CTA pair,
    3 the mixed form (whole rounds, then the rest split) on a grid of 3 CTA pairs (a test form)."""
    _check("awq_debug_set_gemm_split", load_library().awq_debug_set_gemm_split(int(ks)))


class AWQLinear:
    """A quantized linear layer: packed weights plus the per-channel fold scale.

    ``AWQLinear.from_float(W, x_calib)`` runs the whole path on the GPU: the
    activation statistic of ``x_calib`` (a1), the fold and quantizer (a2);
    ``layer(x)`` scales the activations by 1/s and runs the W4A16 kernel
    (a3 for M <= 32, a4 otherwise).
    """

    def __init__(self, qweight, scales, zeros, s, N: int, K: int):
        self.qweight, self.scales, self.zeros, self.s = qweight, scales, zeros, s
        self.N, self.K = N, K

    @classmethod
    def from_float(cls, W, x_calib, alpha: float = 0.5):
        s, _ = awq_activation_scale(x_calib, alpha, want_scaled=False)
        q, sc, z = awq_quantize_g128(W, s)
        return cls(q, sc, z, s, W.shape[0], W.shape[1])

    def __call__(self, x, y=None):
        xs = awq_scale_activations(x, self.s)
        return awq_w4a16_linear(xs, self.qweight, self.scales, self.zeros, self.N, y)


def awq_scale_activations(x, s, x_scaled=None):
    """a1 with a stored s: x' = fp16(x / s) (the activation half of the equivalent transform)."""
    torch = _torch()
    _need(x, torch.float16, "x", 2)
    M, K = x.shape
    if x_scaled is None:
        x_scaled = torch.empty_like(x)
    validate_scale_activations(x, s, x_scaled)
    st = load_library().awq_scale_activations(_ptr(x), _ptr(s), M, K, _ptr(x_scaled), _stream_ptr())
    _check("awq_scale_activations", st)
    return x_scaled


# ---------------------------------------------------------------------------- 8-bit integer linear layers
INT8_MAX_K = 131056


def _check_int8_k(K: int):
    if K < 16 or K % 16 or K > INT8_MAX_K:
        raise ValueError(f"K must be a multiple of 16 in [16, {INT8_MAX_K}], got {K}")


def validate_quantize_rows(x, s, q, step, require_cuda=True, names=("x", "s", "xq", "sx")):
    torch = _torch()
    _need(x, torch.float16, names[0], 2, require_cuda=require_cuda)
    rows, K = x.shape
    if rows < 1:
        raise ValueError(f"{names[0]} must have at least one row")
    _check_int8_k(K)
    if s is not None:
        _check_vec(s, K, names[1], require_cuda)
    _need(q, torch.int8, names[2], 2, require_cuda=require_cuda)
    if tuple(q.shape) != (rows, K):
        raise ValueError(f"{names[2]} must have shape {(rows, K)}, got {tuple(q.shape)}")
    _need(step, torch.float32, names[3], 1, require_cuda=require_cuda)
    if step.numel() != rows:
        raise ValueError(f"{names[3]} must have {rows} elements, got {step.numel()}")


def _quantize_rows(fn_name: str, x, s, out, names):
    torch = _torch()
    _need(x, torch.float16, names[0], 2)
    rows, K = x.shape
    if out is None:
        out = (torch.empty((rows, K), dtype=torch.int8, device=x.device),
               torch.empty(rows, dtype=torch.float32, device=x.device))
    q, step = out
    validate_quantize_rows(x, s, q, step, names=names)
    st = getattr(load_library(), fn_name)(_ptr(x), _ptr(s), rows, K, _ptr(q), _ptr(step), _stream_ptr())
    _check(fn_name, st)
    return q, step


def awq_quantize_tokens(x, s=None, out=None):
    """x' = fp16(x / s) (x itself without s) in 8 bits per token: (xq int8 [M, K], sx fp32 [M])."""
    return _quantize_rows("awq_quantize_tokens", x, s, out, ("x", "s", "xq", "sx"))


def awq_quantize_channels(W, fold_scale=None, out=None):
    """w' = fp16(W * fold_scale) in 8 bits per output channel: (wq int8 [N, K], sw fp32 [N])."""
    return _quantize_rows("awq_quantize_channels", W, fold_scale, out, ("W", "fold_scale", "wq", "sw"))


def validate_w8a8(xq, sx, wq, sw, y, require_cuda=True):
    torch = _torch()
    _need(xq, torch.int8, "xq", 2, require_cuda=require_cuda)
    _need(wq, torch.int8, "wq", 2, require_cuda=require_cuda)
    (M, K), N = xq.shape, wq.shape[0]
    if M < 1 or N < 1:
        raise ValueError("xq and wq must have at least one row")
    if wq.shape[1] != K:
        raise ValueError(f"wq must have K={K} columns, got {wq.shape[1]}")
    _check_int8_k(K)
    _check_vec(sx, M, "sx", require_cuda)
    _check_vec(sw, N, "sw", require_cuda)
    _need(y, torch.float16, "y", 2, require_cuda=require_cuda)
    if tuple(y.shape) != (M, N):
        raise ValueError(f"y must have shape {(M, N)}, got {tuple(y.shape)}")


def awq_w8a8_linear(xq, sx, wq, sw, y=None):
    """y[M, N] = fp16((xq . wq^T) * sx * sw), the integer sums exact (tcgen05 int8)."""
    torch = _torch()
    _need(xq, torch.int8, "xq", 2)
    _need(wq, torch.int8, "wq", 2)
    (M, K), N = xq.shape, wq.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=xq.device)
    validate_w8a8(xq, sx, wq, sw, y)
    st = load_library().awq_w8a8_linear(_ptr(xq), _ptr(sx), _ptr(wq), _ptr(sw), _ptr(y), M, N, K, _stream_ptr())
    _check("awq_w8a8_linear", st)
    return y


class AWQInt8Linear:
    """A linear layer in 8-bit integers: codes and steps per output channel, and the stored scale s
    (or None) that its activations are divided by.

    ``AWQInt8Linear.from_float(W, x_calib)`` takes s from the activation statistic of ``x_calib``
    and quantizes the folded weight; ``layer(x)`` quantizes the tokens and multiplies.
    """

    def __init__(self, wq, sw, s=None):
        torch = _torch()
        _need(wq, torch.int8, "wq", 2)
        self.N, self.K = wq.shape
        if self.N < 1:
            raise ValueError("wq must have at least one row")
        _check_int8_k(self.K)
        _check_vec(sw, self.N, "sw")
        if s is not None:
            _check_vec(s, self.K, "s")
        self.wq, self.sw, self.s = wq, sw, s

    @classmethod
    def from_float(cls, W, x_calib=None, alpha: float = 0.5):
        s = None if x_calib is None else awq_activation_scale(x_calib, alpha, want_scaled=False)[0]
        wq, sw = awq_quantize_channels(W, s)
        return cls(wq, sw, s)

    def __call__(self, x, y=None, workspace=None):
        # the weights were checked when the layer was made; they and x have to be on the current device
        torch = _torch()
        dev = torch.cuda.current_device()
        if (y is None and type(x) is torch.Tensor and x.dtype is torch.float16 and x.dim() == 2 and x.shape[1] == self.K and
                x.shape[0] > 0 and x.get_device() == dev and x.is_contiguous() and self.wq.get_device() == dev):
            return _w8a8_forward(x, self.wq, self.sw, self.s, None, workspace)
        return awq_w8a8_forward(x, self.wq, self.sw, self.s, y, workspace)


def validate_w8a8_forward(x, wq, sw, s, y, require_cuda=True):
    torch = _torch()
    _need(x, torch.float16, "x", 2, require_cuda=require_cuda)
    _need(wq, torch.int8, "wq", 2, require_cuda=require_cuda)
    (M, K), (N, Kw) = x.shape, wq.shape
    if M < 1 or N < 1:
        raise ValueError("x and wq must have at least one row")
    if Kw != K:
        raise ValueError(f"wq must have K={K} columns, got {Kw}")
    _check_int8_k(K)
    _check_vec(sw, N, "sw", require_cuda)
    if s is not None:
        _check_vec(s, K, "s", require_cuda)
    if y is not None:
        _need(y, torch.float16, "y", 2, require_cuda=require_cuda)
        if tuple(y.shape) != (M, N):
            raise ValueError(f"y must have shape {(M, N)}, got {tuple(y.shape)}")


def awq_w8a8_forward(x, wq, sw, s=None, y=None, workspace=None):
    """A whole 8-bit linear layer: awq_quantize_tokens(x, s), then awq_w8a8_linear, in one call.

    ``workspace``: int8, at least awq_w8a8_workspace_bytes(M, K) long, for the tokens' codes and steps;
    allocated here if None. Calls that may overlap on the GPU need workspaces of their own."""
    validate_w8a8_forward(x, wq, sw, s, y)
    return _w8a8_forward(x, wq, sw, s, y, workspace)


def _w8a8_forward(x, wq, sw, s, y, workspace):
    (M, K), N = x.shape, wq.shape[0]
    lib = load_library()
    need = (M * K + 255) // 256 * 256 + 4 * M        # awq_w8a8_workspace_bytes(M, K)
    if workspace is None:
        workspace = wq.new_empty(need)
    elif _need(workspace, wq.dtype, "workspace", 1) is None and workspace.numel() < need:
        raise ValueError(f"workspace must hold {need} bytes")
    if y is None:
        y = x.new_empty(M, N)
    st = lib.awq_w8a8_forward(x.data_ptr(), _ptr(s), wq.data_ptr(), sw.data_ptr(), y.data_ptr(), M, N, K,
                              workspace.data_ptr(), need, _stream_ptr())
    if st:
        _check("awq_w8a8_forward", st)
    return y


# ---------------------------------------------------------------------------- residual update and norms
NORM_MAX_K = 32768
NORM_MAX_ALPHA = 16777216.0


def _overlap(a, b) -> bool:
    """Whether two contiguous tensors share memory (False if one is None)."""
    if a is None or b is None:
        return False
    pa, pb = a.data_ptr(), b.data_ptr()
    return pa < pb + b.numel() * b.element_size() and pb < pa + a.numel() * a.element_size()


def validate_residual_norm(y, residual, weight, post_weight, gate, alpha, eps, s, h, x, require_cuda=True):
    torch = _torch()
    f16 = torch.float16
    _need(y, f16, "y", 2, require_cuda=require_cuda)
    M, K = shape = y.shape
    if M < 1:
        raise ValueError("y must have at least one row")
    if K < 8 or K % 8 or K > NORM_MAX_K:
        raise ValueError(f"K must be a multiple of 8 in [8, {NORM_MAX_K}], got {K}")
    for t, name in ((residual, "residual"), (h, "h"), (x, "x")):
        if t is not None:
            _need(t, f16, name, 2, require_cuda=require_cuda)
            if t.shape != shape:
                raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    _need(weight, f16, "weight", 1, require_cuda=require_cuda)
    if weight.numel() != K:
        raise ValueError(f"weight must have K={K} elements, got {weight.numel()}")
    if post_weight is not None:
        _need(post_weight, f16, "post_weight", 1, require_cuda=require_cuda)
        if post_weight.numel() != K:
            raise ValueError(f"post_weight must have K={K} elements, got {post_weight.numel()}")
    if gate is not None:
        _need(gate, f16, "gate", 2, require_cuda=require_cuda)
        if gate.shape[1] != K or gate.shape[0] < 1 or M % gate.shape[0]:
            raise ValueError(f"gate must have K={K} columns and a number of rows that divides M={M}, "
                             f"got {tuple(gate.shape)}")
    if s is not None:
        _check_vec(s, K, "s", require_cuda)
    for t, name, others in ((h, "h", (x,)), (x, "x", (h,))):
        if t is None:
            continue
        if any(_overlap(t, v) and t.data_ptr() != v.data_ptr() for v in (y, residual)):
            raise ValueError(f"{name} may be y or residual themselves, but not overlap a part of them")
        if any(_overlap(t, v) for v in (*others, gate, post_weight, weight, s)):
            raise ValueError(f"{name} must not overlap the other output, the gate or the weights")
    if not abs(alpha) <= NORM_MAX_ALPHA or not (0.0 <= eps <= 3.0e38):
        raise ValueError(f"alpha must be finite and at most {NORM_MAX_ALPHA:.0f} in magnitude, and eps finite and not negative")


def awq_residual_norm(y, residual, weight, post_weight=None, gate=None, alpha: float = 1.0, eps: float = 1e-6, s=None,
                      out=None, want_h: bool = True):
    """Residual update after a block and RMS norm before the next one; returns (h, x').

    h = residual + alpha * gate * t with t = y, or y normalised and times ``post_weight`` if given;
    x' = rmsnorm(h) * weight / s. ``residual`` may be None (0); ``gate`` is None (1) or [G, K] with G a
    divisor of M: row m uses gate row m // (M // G). ``s`` is the next layer's stored scale.
    ``want_h=False`` leaves h unstored (the first result is None). ``out=(h, x')``: in place with
    ``out=(residual, y)`` (or either of them)."""
    torch = _torch()
    h = x = None
    if out is not None:
        h, x = out
        if x is None:
            raise ValueError("x is always written")
    alpha, eps = float(alpha), float(eps)
    dev, f16 = torch.cuda.current_device(), torch.float16
    fits = (out is None and type(y) is torch.Tensor and y.dtype is f16 and y.dim() == 2 and y.get_device() == dev and
            y.is_contiguous())
    if fits:
        M, K = shape = y.shape
        fits = (0 < M and 8 <= K <= NORM_MAX_K and K % 8 == 0 and _fits(weight, f16, 1, K, dev) and
                (residual is None or (_fits(residual, f16, 2, M * K, dev) and residual.shape == shape)) and
                (s is None or _fits(s, torch.float32, 1, K, dev)) and
                (post_weight is None or _fits(post_weight, f16, 1, K, dev)) and
                (gate is None or (type(gate) is torch.Tensor and _fits(gate, f16, 2, gate.numel(), dev) and
                                  gate.shape[1] == K and gate.shape[0] > 0 and M % gate.shape[0] == 0)) and abs(alpha) <= NORM_MAX_ALPHA and
                0.0 <= eps <= 3.0e38)
    if not fits:
        validate_residual_norm(y, residual, weight, post_weight, gate, alpha, eps, s, h, x)
        M, K = y.shape
    if out is None:
        x = torch.empty_like(y)
        if want_h:
            h = torch.empty_like(y)
    per = M // gate.shape[0] if gate is not None else 1
    st = load_library().awq_residual_norm(y.data_ptr(), _ptr(residual), _ptr(gate), per, _ptr(post_weight),
                                          weight.data_ptr(), _ptr(s), alpha, eps, M, K, _ptr(h), x.data_ptr(),
                                          _stream_ptr(dev))
    if st:
        _check("awq_residual_norm", st)
    return h, x


# ---------------------------------------------------------------------------- mixture of experts
MOE_MAX_TOKENS, MOE_MAX_EXPERTS, MOE_MAX_TOP_K = 32, 512, 16


def _validate_moe_weights(router, gate_up, down, I: int, top_k: int, h_scale, require_cuda=True):
    """Checks the layer's weights; returns (E, K)."""
    torch = _torch()
    _need(router, torch.float16, "router", 2, require_cuda=require_cuda)
    E, K = router.shape
    if not 1 <= E <= MOE_MAX_EXPERTS:
        raise ValueError(f"the number of experts must be in [1, {MOE_MAX_EXPERTS}], got {E}")
    if not 1 <= top_k <= min(E, MOE_MAX_TOP_K):
        raise ValueError(f"top_k must be in [1, {min(E, MOE_MAX_TOP_K)}], got {top_k}")
    if K < GROUP_SIZE or K % GROUP_SIZE or I < GROUP_SIZE or I % GROUP_SIZE:
        raise ValueError("K and I must be positive multiples of 128")
    for packed, what, (N, Kin) in ((gate_up, "gate_up", (2 * I, K)), (down, "down", (K, I))):
        if len(packed) != 3:
            raise ValueError(f"{what} must be (qweight, scales, zeros)")
        qb, sb, zb = _packed_sizes_host(N, Kin)
        for t, dtype, size, name in zip(packed, (torch.int32, torch.float16, torch.uint8), (qb // 4, sb // 2, zb),
                                        ("qweight", "scales", "zeros")):
            _need(t, dtype, f"{what} {name}", 2, require_cuda=require_cuda)
            if tuple(t.shape) != (E, size):
                raise ValueError(f"{what} {name} must have shape {(E, size)}, got {tuple(t.shape)}")
    if h_scale is not None:
        _need(h_scale, torch.float32, "h_scale", 2, require_cuda=require_cuda)
        if tuple(h_scale.shape) != (E, I):
            raise ValueError(f"h_scale must have shape {(E, I)}, got {tuple(h_scale.shape)}")
    return E, K


def _validate_moe_tokens(x, y, E: int, K: int, require_cuda=True):
    torch = _torch()
    _need(x, torch.float16, "x", 2, require_cuda=require_cuda)
    T = x.shape[0]
    if not 1 <= T <= MOE_MAX_TOKENS:
        raise ValueError(f"the number of tokens must be in [1, {MOE_MAX_TOKENS}], got {T}")
    if x.shape[1] != K:
        raise ValueError(f"x must have K={K} columns, got {x.shape[1]}")
    if y is not None:
        _need(y, torch.float16, "y", 2, require_cuda=require_cuda)
        if tuple(y.shape) != (T, K):
            raise ValueError(f"y must have shape {(T, K)}, got {tuple(y.shape)}")


def _moe_call(x, router, gate_up, down, E, K, I, top_k, renormalize, h_scale, y, workspace, need=None):
    torch = _torch()
    lib = load_library()
    T = x.shape[0]
    if need is None:
        need = int(lib.awq_moe_workspace_bytes(T, E, K, I, top_k))
    if need == 0:
        raise ValueError("shape out of range for the mixture-of-experts layer")
    if workspace is None:
        workspace = gate_up[2].new_empty(need)
    else:
        _need(workspace, torch.uint8, "workspace", 1)
        if workspace.numel() < need:
            raise ValueError(f"workspace must hold {need} bytes")
    if y is None:
        y = torch.empty_like(x)
    st = lib.awq_moe_w4a16(x.data_ptr(), router.data_ptr(), gate_up[0].data_ptr(), gate_up[1].data_ptr(),
                           gate_up[2].data_ptr(), down[0].data_ptr(), down[1].data_ptr(), down[2].data_ptr(),
                           _ptr(h_scale), T, E, K, I, top_k, 1 if renormalize else 0, y.data_ptr(),
                           workspace.data_ptr(), need, _stream_ptr())
    if st:
        _check("awq_moe_w4a16", st)
    return y


def awq_moe_w4a16(x, router, gate_up, down, I: int, top_k: int, renormalize: bool = True, h_scale=None, y=None,
                  workspace=None):
    """A whole mixture-of-experts layer for up to 32 tokens: router, top-k, experts, weighted sum.

    x [T, K] fp16; router [E, K] fp16; gate_up and down: (qweight, scales, zeros) with the experts'
    packed arrays stacked along a first dimension (gate_up: 2 I x K layers, I gate rows then I up
    rows; down: K x I); h_scale [E, I] fp32 divides the intermediate (the down layers' s).
    ``workspace``: uint8, at least awq_moe_workspace_bytes(T, E, K, I, top_k) long; allocated here if
    None. Calls that may overlap on the GPU need workspaces of their own."""
    I, top_k = int(I), int(top_k)
    E, K = _validate_moe_weights(router, gate_up, down, I, top_k, h_scale)
    _validate_moe_tokens(x, y, E, K)
    return _moe_call(x, router, gate_up, down, E, K, I, top_k, renormalize, h_scale, y, workspace)


class AWQMoE:
    """A mixture-of-experts layer with packed 4-bit experts (decode, up to 32 tokens a call).

    ``AWQMoE.from_float(router, W_gate_up, W_down, top_k, x_calib)`` takes one scale s for the router
    and the gate/up layers from the activation statistic of ``x_calib`` (they share their input),
    folds and quantizes every expert; ``layer(x)`` scales the activations by 1/s (skipped with
    ``scaled=True``, for an x that awq_residual_norm has already divided) and runs the layer.
    """

    def __init__(self, router, gate_up, down, I: int, top_k: int, renormalize: bool = True, h_scale=None, s=None):
        self.I, self.top_k, self.renormalize = int(I), int(top_k), bool(renormalize)
        self.E, self.K = _validate_moe_weights(router, gate_up, down, self.I, self.top_k, h_scale)
        if s is not None:
            _check_vec(s, self.K, "s")
        self.router, self.gate_up, self.down, self.h_scale, self.s = router, tuple(gate_up), tuple(down), h_scale, s
        self._need = [int(load_library().awq_moe_workspace_bytes(t, self.E, self.K, self.I, self.top_k))
                      for t in range(MOE_MAX_TOKENS + 1)]    # workspace bytes by the number of tokens

    @classmethod
    def from_float(cls, router, W_gate_up, W_down, top_k: int, x_calib=None, alpha: float = 0.5, renormalize: bool = True,
                   h_scale=None):
        """W_gate_up [E, 2 I, K], W_down [E, K, I], router [E, K], all fp16; h_scale [E, I] or None is
        folded into the down layers and divides their input."""
        torch = _torch()
        _need(W_gate_up, torch.float16, "W_gate_up", 3)
        _need(W_down, torch.float16, "W_down", 3)
        E, I2, K = W_gate_up.shape
        if tuple(W_down.shape) != (E, K, I2 // 2) or I2 % 2:
            raise ValueError(f"W_gate_up [E, 2 I, K] and W_down [E, K, I] disagree: {tuple(W_gate_up.shape)}, "
                             f"{tuple(W_down.shape)}")
        s = None
        if x_calib is not None:
            s, _ = awq_activation_scale(x_calib, alpha, want_scaled=False)
            router = (router.float() * s).half()
        stack = lambda layers: tuple(torch.stack(t) for t in zip(*layers))  # noqa: E731
        gate_up = stack([awq_quantize_g128(W_gate_up[e], s) for e in range(E)])
        down = stack([awq_quantize_g128(W_down[e], None if h_scale is None else h_scale[e]) for e in range(E)])
        return cls(router, gate_up, down, I2 // 2, top_k, renormalize, h_scale, s)

    def __call__(self, x, y=None, workspace=None, scaled: bool = False):
        # the weights were checked, on one device, when the layer was made; x has to be on that device
        _need(self.router, _torch().float16, "router", 2)
        _validate_moe_tokens(x, y, self.E, self.K)
        if self.s is not None and not scaled:
            x = awq_scale_activations(x, self.s)
        return _moe_call(x, self.router, self.gate_up, self.down, self.E, self.K, self.I, self.top_k, self.renormalize,
                         self.h_scale, y, workspace, self._need[x.shape[0]])
