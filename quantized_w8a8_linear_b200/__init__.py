"""Python binding of libqlin.so -- a B200 (sm_100a) quantized W8A8 linear layer.

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libqlin.so, called through its C ABI (include/qlin.h) with
ctypes. PyTorch supplies device memory and the current CUDA stream. There is
no CPU fallback: if the library is missing, importing it raises.

Functions keep the C names:

    Wq, s_w = qlin_quantize_weight(W, QLIN_W_INT8_ROW)
    Y = qlin_int8_outlier_forward(X, Wq, s_w, threshold=6.0)
    Wq8, s8 = qlin_quantize_weight(W, QLIN_W_FP8_TENSOR)
    xs = qlin_calibrate_input_scale(X_calibration)
    Y = qlin_fp8_forward(X, Wq8, s8, QLIN_W_FP8_TENSOR, x_scale=xs)

Beside the projections, layer norm (straight to their codes, if wanted) and
low-rank adapters of many requests, with their gradients:

    Xq, s_x = qlin_layer_norm_fp8_prep(X, gamma, beta)
    Y = qlin_fp8_gemm(Xq, s_x, Wq8, s8, QLIN_W_FP8_CHANNEL, X.dtype)
    plan = qlin_lora_plan(adapter_of_row, L)            # once per batch
    qlin_lora_forward(Xn, A, B, scale, plan, Y, H=H)    # Y += s (Xn A^T) B^T, in place
    dX, dA, dB = qlin_lora_backward(dY, Xn, A, B, scale, plan, H, dX=dX)
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlin.so")

QLIN_OK, QLIN_ERR_INVALID_ARG, QLIN_ERR_UNSUPPORTED, QLIN_ERR_ALIGNMENT = 0, 1, 2, 3
QLIN_ERR_WORKSPACE, QLIN_ERR_CUDA, QLIN_ERR_TIMEOUT = 4, 5, 6
QLIN_F16, QLIN_BF16 = 0, 1
QLIN_W_INT8_ROW, QLIN_W_FP8_TENSOR, QLIN_W_FP8_CHANNEL, QLIN_W_INT4_G128, QLIN_W_INT8_BLOCK32 = 0, 1, 2, 3, 4
QLIN_W_NVFP4 = 5
QLIN_OP_INT8_OUTLIER, QLIN_OP_FP8, QLIN_OP_W4A8, QLIN_OP_QUANTIZE_WEIGHT, QLIN_OP_INT8_PREP = 0, 1, 2, 3, 4
QLIN_OP_INT8_BLOCK, QLIN_OP_FP8_GEMM, QLIN_OP_LAYER_NORM_BACKWARD = 5, 6, 7

_STATUS_NAMES = {0: "QLIN_OK", 1: "QLIN_ERR_INVALID_ARG", 2: "QLIN_ERR_UNSUPPORTED", 3: "QLIN_ERR_ALIGNMENT",
                 4: "QLIN_ERR_WORKSPACE", 5: "QLIN_ERR_CUDA", 6: "QLIN_ERR_TIMEOUT"}


class QlinError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python quantized_w8a8_linear_b200/build.py`")
    L = ctypes.CDLL(LIB_PATH)
    P, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    st = ctypes.c_int
    sigs = {
        "qlin_workspace_bytes": (sz, [i32, i64, i64, i64]),
        "qlin_quantize_weight": (st, [P, i32, i64, i64, i32, P, P, P, sz, P]),
        "qlin_calibrate_input_scale": (st, [P, i32, i64, i64, P, P, sz, P]),
        "qlin_int8_outlier_forward": (st, [P, i32, i64, i64, P, P, i64, f32, P, P, P, sz, P]),
        "qlin_fp8_forward": (st, [P, i32, i64, i64, P, P, i32, i64, P, P, P, P, sz, P]),
        "qlin_int8_outlier_prepare": (st, [P, i32, i64, i64, P, P, i64, f32, P, sz, P]),
        "qlin_int8_outlier_forward_noalloc": (st, [P, i32, i64, i64, P, P, i64, f32, P, P, P]),
        "qlin_int8_outlier_gemm": (st, [i32, i64, i64, P, P, i64, P, P, P, sz, P]),
        "qlin_int8_outlier_gemm_i32": (st, [i64, i64, P, i64, P, P, sz, P]),
        "qlin_fp8_gemm": (st, [i32, i64, i64, P, P, P, P, i32, i64, P, P, P, P, sz, P]),
        "qlin_w4a8_forward": (st, [P, i32, i64, i64, P, P, i64, P, P, P, sz, P]),
        "qlin_fp_linear_forward": (st, [P, i32, i64, i64, P, i64, P, P, P]),
        "qlin_fp8_weight_only_forward": (st, [P, i32, i64, i64, P, P, i64, P, P, P]),
        "qlin_nvfp4_weight_only_forward": (st, [P, i32, i64, i64, P, P, i64, P, P, P]),
        "qlin_int8_block_forward": (st, [P, i32, i64, i64, P, P, i64, P, P, P, sz, P]),
        "qlin_int8_block_prep": (st, [P, i32, i64, i64, P, P, P]),
        "qlin_w4a8_gemm": (st, [i32, i64, i64, P, P, P, P, i64, P, P, P]),
        "qlin_w4a8_prep": (st, [P, i32, i64, i64, P, P, P]),
        "qlin_w4a8_group_i32": (st, [P, P, i64, i64, i64, i32, P, P]),
        "qlin_int8_prep": (st, [P, i32, i64, i64, f32, P, P, P, P, P, P, i64, P, sz, P]),
        "qlin_outlier_weights": (st, [P, P, i64, i64, P, P, i32, P, i64, P]),
        "qlin_int8_gemm_i32": (st, [P, P, i64, i64, i64, P, P]),
        "qlin_fp8_prep": (st, [P, i32, i64, i64, P, P, P, P]),
        "qlin_e4m3_encode_f32": (st, [P, P, i64, P]),
        "qlin_layer_norm_forward": (st, [P, i32, i64, i64, P, P, f32, P, P, P, P]),
        "qlin_layer_norm_fp8_prep": (st, [P, i32, i64, i64, P, P, f32, P, P, P, P]),
        "qlin_layer_norm_w4a8_prep": (st, [P, i32, i64, i64, P, P, f32, P, P, P]),
        "qlin_layer_norm_backward": (st, [P, P, i32, i64, i64, P, P, P, P, P, P, P, sz, P]),
        "qlin_lora_plan_bytes": (sz, [i64, i64]),
        "qlin_lora_plan": (st, [P, i64, i64, P, sz, P]),
        "qlin_lora_forward": (st, [P, i32, i64, i64, P, P, P, i64, i64, i64, P, sz, P, P, P]),
        "qlin_lora_forward_h_bytes": (sz, [i64, i64]),
        "qlin_lora_backward_workspace_bytes": (sz, [i64, i64]),
        "qlin_lora_backward": (st, [P, P, i32, i64, i64, P, P, P, i64, i64, i64, P, sz, P, P, P, P, P, sz, P]),
        "qlin_get_device_status": (st, [P, i32]),
        "qlin_set_wait_timeout_ns": (st, [ctypes.c_uint64]),
        "qlin_set_gemm_schedule": (st, [ctypes.c_int]),
        "qlin_debug_inject_wait_timeout": (st, [ctypes.c_int]),
        "qlin_last_error_string": (ctypes.c_char_p, []),
        "qlin_version": (i32, []),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


lib = _load()


def exported_symbols():
    """Names declared in include/qlin.h that this library must export."""
    import re
    hdr = os.path.join(os.path.dirname(_HERE), "include", "qlin.h")
    with open(hdr) as f:
        text = f.read()
    return sorted(set(re.findall(r"^QLIN_API\s+[\w\s\*]+?\b(qlin_\w+)\s*\(", text, flags=re.M)))


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _check(status: int):
    if status != QLIN_OK:
        raise QlinError(status, lib.qlin_last_error_string().decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libqlin takes CUDA tensors (device pointers)")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return QLIN_BF16
    if t.dtype == torch.float16:
        return QLIN_F16
    raise TypeError(f"activations must be fp16 or bf16, got {t.dtype}")


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _tensor(t: Optional[torch.Tensor], name: str, shape: tuple, dtype: torch.dtype, index: int):
    """Pointer of an argument that the kernel reads or writes at this shape, dtype and CUDA device (None: NULL)."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _matrix(t: torch.Tensor, name: str = "X"):
    """(pointer, dtype code, rows, columns, CUDA device index) of a 16-bit matrix."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(t.shape)}")
    M, K = t.shape
    if not t.is_cuda:
        raise ValueError("libqlin takes CUDA tensors (device pointers)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr(), _dt(t), M, K, t.get_device()


def _new(shape: tuple, dtype: torch.dtype, like: torch.Tensor) -> torch.Tensor:
    """An uninitialised contiguous 1-D or 2-D tensor beside `like` (empty_strided: a microsecond less than empty)."""
    return torch.empty_strided(shape, (shape[1], 1) if len(shape) == 2 else (1,), dtype=dtype, device=like.device)


def _call(index: int, fn, *args) -> None:
    """The C call on the tensors' own device and on that device's current stream."""
    if index == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != QLIN_OK:
        _check(status)


_ws_cache = {}


def workspace(op: int, M: int, N: int, K: int, device) -> torch.Tensor:
    """A (cached) device workspace of qlin_workspace_bytes(op, M, N, K) bytes."""
    n = int(lib.qlin_workspace_bytes(op, M, N, K))
    dev = torch.device(device)
    key = (dev.index, op)
    t = _ws_cache.get(key)
    if t is None or t.numel() < n:
        t = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
        _ws_cache[key] = t
    return t


def qlin_workspace_bytes(op: int, M: int, N: int, K: int) -> int:
    return int(lib.qlin_workspace_bytes(op, M, N, K))


# ---------------------------------------------------------------------------
# public API
# ---------------------------------------------------------------------------

def qlin_quantize_weight(W: torch.Tensor, mode: int):
    """Offline weight quantisation. Returns (Wq, w_scale) on W's device."""
    N, K = W.shape
    dev = W.device
    if mode == QLIN_W_INT8_ROW:
        Wq = torch.empty((N, K), dtype=torch.int8, device=dev)
        s = torch.empty((N,), dtype=torch.float32, device=dev)
    elif mode == QLIN_W_FP8_TENSOR:
        Wq = torch.empty((N, K), dtype=torch.uint8, device=dev)
        s = torch.empty((1,), dtype=torch.float32, device=dev)
    elif mode == QLIN_W_FP8_CHANNEL:
        Wq = torch.empty((N, K), dtype=torch.uint8, device=dev)
        s = torch.empty((N, 1), dtype=torch.bfloat16, device=dev)
    elif mode == QLIN_W_INT4_G128:
        Wq = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
        s = torch.empty((N, K // 128), dtype=torch.float32, device=dev)
    elif mode == QLIN_W_INT8_BLOCK32:
        Wq = torch.empty((N, K), dtype=torch.int8, device=dev)
        s = torch.empty((N, K // 32), dtype=torch.float32, device=dev)
    elif mode == QLIN_W_NVFP4:
        Wq = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
        s = torch.empty((nvfp4_scale_offset(N, K) + 4,), dtype=torch.uint8, device=dev)
    else:
        raise ValueError(mode)
    ws = workspace(QLIN_OP_QUANTIZE_WEIGHT, 0, N, K, dev)
    _check(lib.qlin_quantize_weight(_ptr(W), _dt(W), N, K, mode, _ptr(Wq), _ptr(s), _ptr(ws), ws.numel(),
                                    _stream(dev)))
    return Wq, s


def nvfp4_scale_offset(N: int, K: int) -> int:
    """Byte offset of the fp32 tensor scale in a QLIN_W_NVFP4 w_scale buffer
    (after the E4M3 block scales [N, K/16], rounded up to 16 bytes)."""
    return (N * K // 16 + 15) // 16 * 16


def nvfp4_scales(w_scale: torch.Tensor, N: int, K: int):
    """(E4M3 block scales uint8 [N, K/16], fp32 tensor scale [1]) views of a QLIN_W_NVFP4 w_scale buffer."""
    off = nvfp4_scale_offset(N, K)
    return w_scale[: N * K // 16].view(N, K // 16), w_scale[off:off + 4].view(torch.float32)


def qlin_calibrate_input_scale(X: torch.Tensor) -> torch.Tensor:
    """Static FP8 input scale by max calibration: absmax(X) / 448 (device fp32 [1])."""
    M, K = X.shape
    out = torch.empty((1,), dtype=torch.float32, device=X.device)
    ws = workspace(QLIN_OP_QUANTIZE_WEIGHT, M, 0, K, X.device)
    _check(lib.qlin_calibrate_input_scale(_ptr(X), _dt(X), M, K, _ptr(out), _ptr(ws), ws.numel(),
                                          _stream(X.device)))
    return out


def qlin_int8_outlier_forward(X: torch.Tensor, Wq: torch.Tensor, w_scale: torch.Tensor, threshold: float = 6.0,
                              bias: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
                              ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """LLM.int8 linear: Y[M,N] = int8(X \\ O) Wq^T (dequantised) + X[:,O] W_O^T + bias."""
    M, K = X.shape
    N = Wq.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=X.dtype, device=X.device)
    if ws is None:
        ws = workspace(QLIN_OP_INT8_OUTLIER, M, N, K, X.device)
    _check(lib.qlin_int8_outlier_forward(_ptr(X), _dt(X), M, K, _ptr(Wq), _ptr(w_scale), N, float(threshold),
                                         _ptr(bias), _ptr(Y), _ptr(ws), ws.numel(), _stream(X.device)))
    return Y


def qlin_int8_outlier_forward_noalloc(X: torch.Tensor, Wq: torch.Tensor, w_scale: torch.Tensor,
                                      threshold: float = 6.0, bias: Optional[torch.Tensor] = None,
                                      Y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """LLM.int8 linear with the library's built-in scratch (no workspace argument)."""
    M, K = X.shape
    N = Wq.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=X.dtype, device=X.device)
    _check(lib.qlin_int8_outlier_forward_noalloc(_ptr(X), _dt(X), M, K, _ptr(Wq), _ptr(w_scale), N,
                                                 float(threshold), _ptr(bias), _ptr(Y), _stream(X.device)))
    return Y


def qlin_int8_outlier_prepare(X: torch.Tensor, Wq: torch.Tensor, w_scale: torch.Tensor, threshold: float,
                              ws: torch.Tensor) -> None:
    """Stage 1 of the LLM.int8 forward: outlier set, codes, scales, X_O, W_O into `ws`."""
    M, K = X.shape
    N = Wq.shape[0]
    _check(lib.qlin_int8_outlier_prepare(_ptr(X), _dt(X), M, K, _ptr(Wq), _ptr(w_scale), N, float(threshold),
                                         _ptr(ws), ws.numel(), _stream(X.device)))


def qlin_int8_outlier_gemm(dtype: torch.dtype, M: int, K: int, Wq: torch.Tensor, w_scale: torch.Tensor,
                           Y: torch.Tensor, ws: torch.Tensor, bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Stage 2 of the LLM.int8 forward: tcgen05 GEMM + fused epilogue, reading `ws`."""
    N = Wq.shape[0]
    dt = QLIN_BF16 if dtype == torch.bfloat16 else QLIN_F16
    _check(lib.qlin_int8_outlier_gemm(dt, M, K, _ptr(Wq), _ptr(w_scale), N, _ptr(bias), _ptr(Y), _ptr(ws),
                                      ws.numel(), _stream(Wq.device)))
    return Y


def qlin_int8_outlier_gemm_i32(M: int, K: int, Wq: torch.Tensor, ws: torch.Tensor) -> torch.Tensor:
    """int32 accumulator of the LLM.int8 GEMM without the outlier columns, from
    the workspace a prepare call filled (parity export of the same kernel)."""
    N = Wq.shape[0]
    C = torch.empty((M, N), dtype=torch.int32, device=Wq.device)
    _check(lib.qlin_int8_outlier_gemm_i32(M, K, _ptr(Wq), N, _ptr(C), _ptr(ws), ws.numel(), _stream(Wq.device)))
    return C


def qlin_fp8_gemm(Xq: torch.Tensor, s_x: Optional[torch.Tensor], Wq: torch.Tensor, w_scale: torch.Tensor,
                  wmode: int, dtype: torch.dtype, x_scale: Optional[torch.Tensor] = None,
                  bias: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
                  ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """GEMM stage of the FP8 forward on codes from qlin_fp8_prep. ws: optional
    scratch of workspace(QLIN_OP_FP8_GEMM, ...) bytes (lets the GEMM split
    tiles along K across CTAs); None: whole tiles only."""
    M, K = Xq.shape
    N = Wq.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=dtype, device=Xq.device)
    dt = QLIN_BF16 if dtype == torch.bfloat16 else QLIN_F16
    _check(lib.qlin_fp8_gemm(dt, M, K, _ptr(Xq), _ptr(s_x), _ptr(Wq), _ptr(w_scale), wmode, N, _ptr(x_scale),
                             _ptr(bias), _ptr(Y), _ptr(ws), 0 if ws is None else ws.numel(), _stream(Xq.device)))
    return Y


def qlin_fp8_forward(X: torch.Tensor, Wq: torch.Tensor, w_scale: torch.Tensor, wmode: int,
                     x_scale: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                     Y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """FP8 E4M3 W8A8 linear (static per-tensor or dynamic per-token / per-channel scales)."""
    M, K = X.shape
    N = Wq.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=X.dtype, device=X.device)
    if ws is None:
        ws = workspace(QLIN_OP_FP8, M, N, K, X.device)
    _check(lib.qlin_fp8_forward(_ptr(X), _dt(X), M, K, _ptr(Wq), _ptr(w_scale), wmode, N, _ptr(x_scale),
                                _ptr(bias), _ptr(Y), _ptr(ws), ws.numel(), _stream(X.device)))
    return Y


def qlin_w4a8_forward(X: torch.Tensor, Wq4: torch.Tensor, w_scale: torch.Tensor,
                      bias: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """W4A8 linear: int4 per-group-128 weights, per-token int8 activations."""
    M, K = X.shape
    N = Wq4.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=X.dtype, device=X.device)
    if ws is None:
        ws = workspace(QLIN_OP_W4A8, M, N, K, X.device)
    _check(lib.qlin_w4a8_forward(_ptr(X), _dt(X), M, K, _ptr(Wq4), _ptr(w_scale), N, _ptr(bias), _ptr(Y),
                                 _ptr(ws), ws.numel(), _stream(X.device)))
    return Y


def qlin_fp_linear_forward(X: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None,
                           Y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Unquantised 16-bit linear Y = X W^T + bias (X, W, bias in one dtype), tcgen05 kind::f16."""
    M, K = X.shape
    N = W.shape[0]
    if W.dtype != X.dtype or (bias is not None and bias.dtype != X.dtype):
        raise TypeError("X, W and bias must share one 16-bit dtype")
    if Y is None:
        Y = torch.empty((M, N), dtype=X.dtype, device=X.device)
    _check(lib.qlin_fp_linear_forward(_ptr(X), _dt(X), M, K, _ptr(W), N, _ptr(bias), _ptr(Y), _stream(X.device)))
    return Y


def qlin_fp8_weight_only_forward(X: torch.Tensor, Wq: torch.Tensor, w_scale: torch.Tensor,
                                 bias: Optional[torch.Tensor] = None,
                                 Y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Weight-only FP8 linear: Y = X (bf16(decode(Wq) * w_scale))^T + bias, bf16 activations."""
    M, K = X.shape
    N = Wq.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=X.dtype, device=X.device)
    _check(lib.qlin_fp8_weight_only_forward(_ptr(X), _dt(X), M, K, _ptr(Wq), _ptr(w_scale), N, _ptr(bias), _ptr(Y),
                                            _stream(X.device)))
    return Y


def qlin_nvfp4_weight_only_forward(X: torch.Tensor, Wq: torch.Tensor, w_scale: torch.Tensor,
                                   bias: Optional[torch.Tensor] = None,
                                   Y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """NVFP4 weight-only linear: Y = s_t * X (e2m1(code) * e4m3(s_b))^T + bias, bf16 activations."""
    M, K = X.shape
    N = Wq.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=X.dtype, device=X.device)
    _check(lib.qlin_nvfp4_weight_only_forward(_ptr(X), _dt(X), M, K, _ptr(Wq), _ptr(w_scale), N, _ptr(bias),
                                              _ptr(Y), _stream(X.device)))
    return Y


def qlin_int8_block_forward(X: torch.Tensor, Wq: torch.Tensor, w_scale: torch.Tensor,
                            bias: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
                            ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Block-scaled int8 linear: one fp32 weight scale per 32 weights of a row, per-token int8 activations."""
    M, K = X.shape
    N = Wq.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=X.dtype, device=X.device)
    if ws is None:
        ws = workspace(QLIN_OP_INT8_BLOCK, M, N, K, X.device)
    _check(lib.qlin_int8_block_forward(_ptr(X), _dt(X), M, K, _ptr(Wq), _ptr(w_scale), N, _ptr(bias), _ptr(Y),
                                       _ptr(ws), ws.numel(), _stream(X.device)))
    return Y


def qlin_int8_block_prep(X: torch.Tensor):
    """Activation stage of the block-scaled int8 forward: int8 codes as fp16 values [M,K] and s_x [M]."""
    M, K = X.shape
    Xq16 = torch.empty((M, K), dtype=torch.float16, device=X.device)
    s_x = torch.empty((M,), dtype=torch.float32, device=X.device)
    _check(lib.qlin_int8_block_prep(_ptr(X), _dt(X), M, K, _ptr(Xq16), _ptr(s_x), _stream(X.device)))
    return Xq16, s_x


def qlin_w4a8_prep(X: torch.Tensor, Xq: Optional[torch.Tensor] = None, s_x: Optional[torch.Tensor] = None):
    """Activation stage of the W4A8 forward: per-token int8 codes and fp32 scales."""
    M, K = X.shape
    if Xq is None:
        Xq = torch.empty((M, K), dtype=torch.int8, device=X.device)
    if s_x is None:
        s_x = torch.empty((M,), dtype=torch.float32, device=X.device)
    _check(lib.qlin_w4a8_prep(_ptr(X), _dt(X), M, K, _ptr(Xq), _ptr(s_x), _stream(X.device)))
    return Xq, s_x


def qlin_w4a8_gemm(Xq: torch.Tensor, s_x: torch.Tensor, Wq4: torch.Tensor, w_scale: torch.Tensor,
                   dtype: torch.dtype, bias: Optional[torch.Tensor] = None,
                   Y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """GEMM stage of the W4A8 forward on int8 codes and per-token scales."""
    M, K = Xq.shape
    N = Wq4.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=dtype, device=Xq.device)
    dt = QLIN_BF16 if dtype == torch.bfloat16 else QLIN_F16
    _check(lib.qlin_w4a8_gemm(dt, M, K, _ptr(Xq), _ptr(s_x), _ptr(Wq4), _ptr(w_scale), N, _ptr(bias), _ptr(Y),
                              _stream(Xq.device)))
    return Y


def qlin_w4a8_group_i32(Xq: torch.Tensor, Wq4: torch.Tensor, group: int) -> torch.Tensor:
    """int32 partials C_g [M,N] of one group, as the W4A8 GEMM computes them (parity export)."""
    M, K = Xq.shape
    N = Wq4.shape[0]
    C = torch.empty((M, N), dtype=torch.int32, device=Xq.device)
    _check(lib.qlin_w4a8_group_i32(_ptr(Xq), _ptr(Wq4), M, N, K, int(group), _ptr(C), _stream(Xq.device)))
    return C


def qlin_int8_prep(X: torch.Tensor, threshold: float = 6.0):
    """LLM.int8 activation prep alone (parity export). Returns a dict of device tensors."""
    M, K = X.shape
    dev = X.device
    ostride = (K + 7) // 8 * 8
    Xq = torch.empty((M, K), dtype=torch.int8, device=dev)
    s_x = torch.empty((M,), dtype=torch.float32, device=dev)
    flags = torch.empty(((K + 31) // 32,), dtype=torch.int32, device=dev)
    O = torch.empty((K,), dtype=torch.int32, device=dev)
    count = torch.empty((1,), dtype=torch.int32, device=dev)
    X_O = torch.zeros((M, ostride), dtype=X.dtype, device=dev)
    ws = workspace(QLIN_OP_INT8_PREP, M, 0, K, dev)
    _check(lib.qlin_int8_prep(_ptr(X), _dt(X), M, K, float(threshold), _ptr(Xq), _ptr(s_x), _ptr(flags), _ptr(O),
                              _ptr(count), _ptr(X_O), ostride, _ptr(ws), ws.numel(), _stream(dev)))
    return dict(Xq=Xq, s_x=s_x, flags=flags, O=O, count=count, X_O=X_O, ostride=ostride)


def qlin_outlier_weights(Wq: torch.Tensor, w_scale: torch.Tensor, O: torch.Tensor, count: torch.Tensor,
                         dtype: torch.dtype) -> torch.Tensor:
    """W_O [N, round_up(K,8)] = dtype(fp32(Wq[:,O]) * w_scale) (parity export)."""
    N, K = Wq.shape
    ostride = (K + 7) // 8 * 8
    W_O = torch.zeros((N, ostride), dtype=dtype, device=Wq.device)
    dt = QLIN_BF16 if dtype == torch.bfloat16 else QLIN_F16
    _check(lib.qlin_outlier_weights(_ptr(Wq), _ptr(w_scale), N, K, _ptr(O), _ptr(count), dt, _ptr(W_O), ostride,
                                    _stream(Wq.device)))
    return W_O


def qlin_int8_gemm_i32(Xq: torch.Tensor, Wq: torch.Tensor) -> torch.Tensor:
    """Raw tcgen05 int8 GEMM: C[M,N] int32 = Xq Wq^T (parity export)."""
    M, K = Xq.shape
    N = Wq.shape[0]
    C = torch.empty((M, N), dtype=torch.int32, device=Xq.device)
    _check(lib.qlin_int8_gemm_i32(_ptr(Xq), _ptr(Wq), M, N, K, _ptr(C), _stream(Xq.device)))
    return C


def qlin_fp8_prep(X: torch.Tensor, x_scale: Optional[torch.Tensor] = None):
    """FP8 activation codes (uint8 e4m3 [M,K]) and, in dynamic mode, per-token scales."""
    M, K = X.shape
    Xq = torch.empty((M, K), dtype=torch.uint8, device=X.device)
    s_x = torch.empty((M,), dtype=torch.float32, device=X.device)
    _check(lib.qlin_fp8_prep(_ptr(X), _dt(X), M, K, _ptr(x_scale), _ptr(Xq), _ptr(s_x), _stream(X.device)))
    return Xq, s_x


def qlin_e4m3_encode_f32(t: torch.Tensor, codes: Optional[torch.Tensor] = None) -> torch.Tensor:
    """E4M3 codes of fp32 values with the device conversion the FP8 kernels use (parity export)."""
    t = t.reshape(-1)
    if codes is None:
        codes = torch.empty(t.shape, dtype=torch.uint8, device=t.device)
    _check(lib.qlin_e4m3_encode_f32(_ptr(t), _ptr(codes), t.numel(), _stream(t.device)))
    return codes


def qlin_layer_norm_forward(X: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
                            eps: float = 1e-6, Y: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
                            rstd: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Layer norm of the rows of X [M,K]. mean, rstd: fp32 [M] to fill for the backward pass. Y may be X."""
    x, dt, M, K, dev = _matrix(X)
    if Y is None:
        Y = torch.empty_like(X)
    _call(dev, lib.qlin_layer_norm_forward, x, dt, M, K, _tensor(gamma, "gamma", (K,), X.dtype, dev),
          _tensor(beta, "beta", (K,), X.dtype, dev), eps, _tensor(Y, "Y", (M, K), X.dtype, dev),
          _tensor(mean, "mean", (M,), torch.float32, dev), _tensor(rstd, "rstd", (M,), torch.float32, dev))
    return Y


def qlin_layer_norm_fp8_prep(X: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
                             eps: float = 1e-6, x_scale: Optional[torch.Tensor] = None):
    """Layer norm as FP8 codes (uint8 e4m3 [M,K]) and, in dynamic mode, per-token scales [M] for qlin_fp8_gemm."""
    x, dt, M, K, dev = _matrix(X)
    Xq = _new((M, K), torch.uint8, X)
    s_x = _new((M,), torch.float32, X) if x_scale is None else None
    if x_scale is not None:
        x_scale = x_scale.reshape(-1)
    _call(dev, lib.qlin_layer_norm_fp8_prep, x, dt, M, K, _tensor(gamma, "gamma", (K,), X.dtype, dev),
          _tensor(beta, "beta", (K,), X.dtype, dev), eps, _tensor(x_scale, "x_scale", (1,), torch.float32, dev),
          Xq.data_ptr(), None if s_x is None else s_x.data_ptr())
    return Xq, s_x


def qlin_layer_norm_w4a8_prep(X: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
                              eps: float = 1e-6):
    """Layer norm as int8 codes [M,K] and per-token scales [M] for qlin_w4a8_gemm."""
    x, dt, M, K, dev = _matrix(X)
    Xq = _new((M, K), torch.int8, X)
    s_x = _new((M,), torch.float32, X)
    _call(dev, lib.qlin_layer_norm_w4a8_prep, x, dt, M, K, _tensor(gamma, "gamma", (K,), X.dtype, dev),
          _tensor(beta, "beta", (K,), X.dtype, dev), eps, Xq.data_ptr(), s_x.data_ptr())
    return Xq, s_x


def qlin_layer_norm_backward(dY: torch.Tensor, X: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                             gamma: Optional[torch.Tensor] = None, beta_grad: Optional[bool] = None,
                             dX: Optional[torch.Tensor] = None):
    """(dX, dgamma, dbeta) of qlin_layer_norm_forward; dgamma is None without gamma, and dbeta goes with it
    unless beta_grad says otherwise. dX may be dY or X."""
    x, dt, M, K, dev = _matrix(X)
    if beta_grad is None:
        beta_grad = gamma is not None
    if dX is None:
        dX = torch.empty_like(X)
    dgamma = torch.empty_like(gamma) if gamma is not None else None
    dbeta = _new((K,), X.dtype, X) if beta_grad else None
    ws, n = None, 0
    if dgamma is not None or dbeta is not None:
        n = max(_workspace_size(QLIN_OP_LAYER_NORM_BACKWARD, M, 0, K), 16)
        ws = _new((n,), torch.uint8, X)   # its own: calls on other streams have theirs
    _call(dev, lib.qlin_layer_norm_backward, _tensor(dY, "dY", (M, K), X.dtype, dev), x, dt, M, K,
          _tensor(gamma, "gamma", (K,), X.dtype, dev), _tensor(mean, "mean", (M,), torch.float32, dev),
          _tensor(rstd, "rstd", (M,), torch.float32, dev), _tensor(dX, "dX", (M, K), X.dtype, dev),
          None if dgamma is None else dgamma.data_ptr(), None if dbeta is None else dbeta.data_ptr(),
          None if ws is None else ws.data_ptr(), n)
    return dX, dgamma, dbeta


@functools.lru_cache(maxsize=4096)
def _workspace_size(op: int, M: int, N: int, K: int) -> int:
    return int(lib.qlin_workspace_bytes(op, M, N, K))


@functools.lru_cache(maxsize=4096)
def _plan_size(M: int, L: int) -> int:
    return max(int(lib.qlin_lora_plan_bytes(M, L)), 16)


@functools.lru_cache(maxsize=4096)
def _lora_needs_h(M: int, R: int) -> bool:
    return int(lib.qlin_lora_forward_h_bytes(M, R)) > 0


@functools.lru_cache(maxsize=4096)
def _lora_backward_size(M: int, R: int) -> int:
    return max(int(lib.qlin_lora_backward_workspace_bytes(M, R)), 16)


def qlin_lora_plan(idx: torch.Tensor, L: int) -> torch.Tensor:
    """The rows of a batch sorted by adapter, for the calls below. idx int32 [M]: the adapter of each row, or a
    value outside 0..L-1 for a row without one. Made once per batch, used by every projection it passes through."""
    if idx.dim() != 1 or idx.dtype != torch.int32:
        raise TypeError("idx must be a 1-D int32 tensor")
    M, L = idx.shape[0], int(L)
    x = _ptr(idx)
    plan = _new((_plan_size(M, L),), torch.uint8, idx)
    _call(idx.get_device(), lib.qlin_lora_plan, x, M, L, plan.data_ptr(), plan.numel())
    return plan


def _lora_args(M, K, dtype, dev, A, B, scale, plan):
    """(R, N, the C arguments from A to plan_bytes)"""
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError("A must be [L, R, K] and B [L, N, R]")
    L, R, _ = A.shape
    N = B.shape[1]
    size = _plan_size(M, L)
    if plan.numel() != size:
        raise ValueError(f"plan was not made for {M} rows and {L} adapters")
    return R, N, (_tensor(A, "A", (L, R, K), dtype, dev), _tensor(B, "B", (L, N, R), dtype, dev),
                  _tensor(scale, "scale", (L,), torch.float32, dev), L, R, N,
                  _tensor(plan, "plan", (size,), torch.uint8, dev), size)


def qlin_lora_forward(X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor, plan: torch.Tensor,
                      Y: torch.Tensor, H: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Adapters beside a projection, in place: Y[i] += scale[a] * (X[i] A[a]^T) B[a]^T for rows with an adapter.
    H: fp32 [M,R] to fill with X A^T for the backward pass (rows without an adapter are left as they were)."""
    x, dt, M, K, dev = _matrix(X)
    R, N, args = _lora_args(M, K, X.dtype, dev, A, B, scale, plan)
    if H is None and _lora_needs_h(M, R):
        H = _new((M, R), torch.float32, X)
    _call(dev, lib.qlin_lora_forward, x, dt, M, K, *args, _tensor(H, "H", (M, R), torch.float32, dev),
          _tensor(Y, "Y", (M, N), X.dtype, dev))
    return Y


def qlin_lora_backward(dY: torch.Tensor, X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor,
                       plan: torch.Tensor, H: torch.Tensor, dX: Optional[torch.Tensor] = None):
    """(dX, dA, dB) of qlin_lora_forward, bf16. dX: the projection's own input gradient, added to in place
    (None: not computed)."""
    x, dt, M, K, dev = _matrix(X)
    R, N, args = _lora_args(M, K, X.dtype, dev, A, B, scale, plan)
    dA, dB = torch.empty_like(A), torch.empty_like(B)
    n = _lora_backward_size(M, R)
    ws = _new((n,), torch.uint8, X)   # its own: calls on other streams have theirs
    _call(dev, lib.qlin_lora_backward, _tensor(dY, "dY", (M, N), X.dtype, dev), x, dt, M, K, *args,
          _tensor(H, "H", (M, R), torch.float32, dev), _tensor(dX, "dX", (M, K), X.dtype, dev), dA.data_ptr(),
          dB.data_ptr(), ws.data_ptr(), n)
    return dX, dA, dB


def qlin_get_device_status(reset: bool = False) -> int:
    v = ctypes.c_int32(0)
    _check(lib.qlin_get_device_status(ctypes.byref(v), 1 if reset else 0))
    return int(v.value)


def qlin_set_wait_timeout_ns(ns: int) -> None:
    _check(lib.qlin_set_wait_timeout_ns(int(ns)))


def qlin_debug_inject_wait_timeout(on: bool) -> None:
    """Test switch: later launches of tcgen05 kernels wait once on a barrier nothing arrives on (bounded)."""
    _check(lib.qlin_debug_inject_wait_timeout(1 if on else 0))


def qlin_set_gemm_schedule(mode: int) -> None:
    """0 automatic, 1 whole tiles only, 2 stream-K wherever possible (int8 GEMMs)."""
    _check(lib.qlin_set_gemm_schedule(int(mode)))


__all__ = [n for n in dir() if n.startswith(("qlin_", "QLIN_"))] + ["QlinError", "workspace", "lib"]
