"""Python binding of the MI355X FP8-optimizer-state AdamW step.

Argument marshalling only: every call hands raw device pointers of torch
tensors and torch's current HIP stream to ``libcoat_fp8.so`` (the C ABI in
``include/coat_fp8.h``); all arithmetic runs in the HIP kernels. There is no
fallback: if the library is missing or no GPU is present the calls raise.

Method: COAT's optimizer over FP8-compressed Adam state with per-group
dynamic range expansion ("COAT: FP8 training, 40% less memory, 1.4x faster",
blob.wenxiaobai.com, sections "FP8 optimizer states" and "Solution: dynamic
range expansion").
"""
from __future__ import annotations

import ctypes
import json
import os
from dataclasses import dataclass
from typing import Dict, List, Optional, Sequence

import torch

FMT_E4M3 = 0
FMT_E5M2 = 1
FMT_MX4 = 2
FMT_NO_EXPAND = 0x100

COAT_OK, COAT_EINVAL, COAT_EALIGN, COAT_EHIP, COAT_ERANGE = 0, -1, -2, -3, -4
STATIC_MAX_TENSORS = 4096

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcoat_fp8.so")


class CoatError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {strerror(status)} (status {status})")


class _Tensor(ctypes.Structure):
    _fields_ = [("params", ctypes.c_void_p), ("params_bf16", ctypes.c_void_p),
                ("grads", ctypes.c_void_p), ("m_q", ctypes.c_void_p), ("m_s", ctypes.c_void_p),
                ("m_k", ctypes.c_void_p), ("v_q", ctypes.c_void_p), ("v_s", ctypes.c_void_p),
                ("v_k", ctypes.c_void_p), ("n", ctypes.c_int64)]


class _Border(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("rows_per_gate", ctypes.c_int64),
                ("eps", ctypes.c_float), ("scale", ctypes.c_float), ("post", ctypes.c_int32),
                ("stream_type", ctypes.c_int32), ("param_type", ctypes.c_int32), ("grad_type", ctypes.c_int32)]


class _Plan(ctypes.Structure):
    _fields_ = [("workspace", ctypes.c_void_p), ("count", ctypes.c_int32),
                ("tiles", ctypes.c_int64), ("n_total", ctypes.c_int64), ("n_partial", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libcoat_fp8.so (after torch, so both share one HIP runtime)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run python -m fp8_optimizer_state_amd._build")
    L = ctypes.CDLL(LIB_PATH)
    P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    hyper = [f32, f32, f32, f32, f32, i64]
    L.coat_fp8_adamw_step.argtypes = [P, P, P, P, P, P, P, P, P, i64, i32, i32, i32, *hyper, P]
    L.coat_multi_workspace_bytes.argtypes = [i32]
    L.coat_multi_workspace_bytes.restype = ctypes.c_size_t
    L.coat_multi_plan_init.argtypes = [ctypes.POINTER(_Plan), ctypes.POINTER(_Tensor), i32, P,
                                       ctypes.c_size_t, P]
    L.coat_fp8_adamw_step_planned.argtypes = [ctypes.POINTER(_Plan), i32, i32, i32, *hyper, P]
    L.coat_fp8_adamw_step_multi.argtypes = [ctypes.POINTER(_Tensor), i32, i32, i32, i32, *hyper,
                                            P, ctypes.c_size_t, P]
    L.coat_fp8_adamw_step_multi_static.argtypes = [ctypes.POINTER(_Tensor), i32, i32, i32, i32, *hyper, P]
    L.coat_fp8_quantize.argtypes = [P, i64, i32, i32, P, P, P, P]
    L.coat_fp8_dequantize.argtypes = [P, P, P, i64, i32, i32, P, P]
    L.coat_fp8_encode.argtypes = [P, i64, i32, P, P]
    L.coat_fp8_decode.argtypes = [P, i64, i32, P, P]
    L.coat_fp8_act_quantize.argtypes = [P, i64, i32, i32, P, P, P]
    L.coat_fp8_act_dequantize.argtypes = [P, P, i64, i32, i32, P, P]
    L.coat_mx4_code_bytes.argtypes = [i64]
    L.coat_mx4_scale_bytes.argtypes = [i64]
    L.coat_mx4_quantize.argtypes = [P, i64, i64, i64, i32, P, P, P, P, P]
    L.coat_mx4_dequantize.argtypes = [P, P, i64, i64, P, i64, i32, P]
    L.coat_mx4_matmul_workspace_bytes.argtypes = [i64, i64, i64]
    L.coat_mx4_matmul.argtypes = [P, P, i64, P, P, i64, i64, P, i64, i32, P, ctypes.c_size_t, P]
    border = ctypes.POINTER(_Border)
    L.coat_block_norm.argtypes = [border, P, P, P, P, P, P, P, P, P, i32, i32, P]
    L.coat_block_norm_backward_workspace_bytes.argtypes = [border]
    L.coat_block_norm_backward.argtypes = [border, P, P, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    for name in ("coat_mx4_code_bytes", "coat_mx4_scale_bytes"):
        getattr(L, name).restype = i64
    for name in ("coat_mx4_matmul_workspace_bytes", "coat_block_norm_backward_workspace_bytes"):
        getattr(L, name).restype = ctypes.c_size_t
    L.coat_strerror.argtypes = [ctypes.c_int]
    L.coat_strerror.restype = ctypes.c_char_p
    L.coat_abi_version.restype = ctypes.c_int
    for name in ("coat_fp8_adamw_step", "coat_multi_plan_init", "coat_fp8_adamw_step_planned",
                 "coat_fp8_adamw_step_multi", "coat_fp8_adamw_step_multi_static", "coat_fp8_quantize", "coat_fp8_dequantize",
                 "coat_fp8_encode", "coat_fp8_decode", "coat_fp8_act_quantize",
                 "coat_fp8_act_dequantize", "coat_mx4_quantize", "coat_mx4_dequantize", "coat_mx4_matmul",
                 "coat_block_norm", "coat_block_norm_backward"):
        getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def strerror(status: int) -> str:
    return lib().coat_strerror(status).decode()


def _check(status: int, what: str):
    if status != COAT_OK:
        raise CoatError(status, what)


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _ptr(t: Optional[torch.Tensor], dtype: torch.dtype, numel: int, name: str):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    return t.data_ptr()


def ngroups(n: int, group: int) -> int:
    return (n + group - 1) // group


# ---------------------------------------------------------------- single tensor

def adamw_step(params, params_bf16, grads, m_q, m_s, m_k, v_q, v_s, v_k, *, group: int,
               fmt_m: int, fmt_v: int, lr: float, beta1: float, beta2: float, eps: float,
               weight_decay: float, step: int, stream=None) -> None:
    """One FP8-state AdamW step of one tensor, in place (asynchronous)."""
    n = params.numel()
    ng = ngroups(n, group)
    rc = lib().coat_fp8_adamw_step(
        _ptr(params, torch.float32, n, "params"), _ptr(params_bf16, torch.bfloat16, n, "params_bf16"),
        _ptr(grads, torch.bfloat16, n, "grads"),
        _ptr(m_q, torch.uint8, n, "m_q"), _ptr(m_s, torch.float64, ng, "m_s"),
        _ptr(m_k, torch.float32, ng, "m_k"),
        _ptr(v_q, torch.uint8, n, "v_q"), _ptr(v_s, torch.float64, ng, "v_s"),
        _ptr(v_k, torch.float32, ng, "v_k"),
        n, group, fmt_m, fmt_v, lr, beta1, beta2, eps, weight_decay, step, _stream(stream))
    _check(rc, "coat_fp8_adamw_step")


# ---------------------------------------------------------------- codec

def quantize(x, q, s, k, *, group: int, fmt: int, stream=None) -> None:
    n = x.numel()
    ng = ngroups(n, group)
    rc = lib().coat_fp8_quantize(_ptr(x, torch.float32, n, "x"), n, group, fmt,
                                 _ptr(q, torch.uint8, n, "q"), _ptr(s, torch.float64, ng, "s"),
                                 _ptr(k, torch.float32, ng, "k"), _stream(stream))
    _check(rc, "coat_fp8_quantize")


def dequantize(q, s, k, x, *, group: int, fmt: int, stream=None) -> None:
    n = q.numel()
    ng = ngroups(n, group)
    rc = lib().coat_fp8_dequantize(_ptr(q, torch.uint8, n, "q"), _ptr(s, torch.float64, ng, "s"),
                                   _ptr(k, torch.float32, ng, "k"), n, group, fmt,
                                   _ptr(x, torch.float32, n, "x"), _stream(stream))
    _check(rc, "coat_fp8_dequantize")


def encode(y, q, *, fmt: int, stream=None) -> None:
    n = y.numel()
    rc = lib().coat_fp8_encode(_ptr(y, torch.float32, n, "y"), n, fmt,
                               _ptr(q, torch.uint8, n, "q"), _stream(stream))
    _check(rc, "coat_fp8_encode")


def decode(q, y, *, fmt: int, stream=None) -> None:
    n = q.numel()
    rc = lib().coat_fp8_decode(_ptr(q, torch.uint8, n, "q"), n, fmt,
                               _ptr(y, torch.float32, n, "y"), _stream(stream))
    _check(rc, "coat_fp8_decode")


def act_nscales(n: int, group: int) -> int:
    """Scales of an activation tensor: one per tensor (group 0) or per group."""
    return 1 if group == 0 else ngroups(n, group)


def act_quantize(x, q, scale, *, group: int, fmt: int, stream=None) -> None:
    """bf16 activations -> FP8 codes + fp32 scales, per tensor (group 0) or per group."""
    n = x.numel()
    rc = lib().coat_fp8_act_quantize(_ptr(x, torch.bfloat16, n, "x"), n, group, fmt,
                                     _ptr(q, torch.uint8, n, "q"),
                                     _ptr(scale, torch.float32, act_nscales(n, group), "scale"),
                                     _stream(stream))
    _check(rc, "coat_fp8_act_quantize")


def act_dequantize(q, scale, x, *, group: int, fmt: int, stream=None) -> None:
    """FP8 codes + fp32 scales -> bf16 activations."""
    n = q.numel()
    rc = lib().coat_fp8_act_dequantize(_ptr(q, torch.uint8, n, "q"),
                                       _ptr(scale, torch.float32, act_nscales(n, group), "scale"), n,
                                       group, fmt, _ptr(x, torch.bfloat16, n, "x"), _stream(stream))
    _check(rc, "coat_fp8_act_dequantize")


# ---------------------------------------------------------------- layer-input operators
#
# These work on (rows, channels) matrices, on the device that holds them: the
# calls take `stream`, or that device's current stream, and may be made while
# another device is current.

_TYPES = {torch.bfloat16: 0, torch.float32: 1}


def _float_type(t: torch.Tensor, name: str) -> int:
    kind = _TYPES.get(t.dtype)
    if kind is None:
        raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return kind


def _operand(t: torch.Tensor, dtype: torch.dtype, shape, gpu: int, name: str) -> int:
    """Address of a tensor without gaps that has this type and shape and is on GPU `gpu`."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == gpu and t.is_contiguous():
        return t.data_ptr()
    if t.get_device() != gpu:
        raise ValueError(f"{name} must be on GPU {gpu} like the other tensors, got {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _gpu_of(t: torch.Tensor, name: str) -> int:
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got {t.dim()} dimensions")
    gpu = t.get_device()
    if gpu < 0 or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return gpu


def _row_stride(t: torch.Tensor, name: str) -> int:
    """Elements from row to row of a matrix whose rows have no gaps."""
    rows, cols = t.shape
    ld, step = t.stride()
    if rows > 1 and ld < cols or cols > 1 and step != 1:
        raise ValueError(f"{name} must have rows without gaps, got strides {t.stride()}")
    return ld if rows > 1 else max(cols, 1)


# torch.cuda.current_stream() builds a Stream object: 2 us, a fifth of a small call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda gpu: torch.cuda.current_stream(gpu).cuda_stream)
_current_gpu = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device  # of a process that has GPU tensors


def _call(gpu: int, stream, function, what: str, *args) -> None:
    """function(*args, stream handle), with GPU `gpu` current."""
    if stream is not None and stream.device_index != gpu:
        raise ValueError(f"the stream belongs to GPU {stream.device_index}, the tensors are on GPU {gpu}")
    if gpu == _current_gpu():
        rc = function(*args, _raw_stream(gpu) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(gpu):
            rc = function(*args, _raw_stream(gpu) if stream is None else stream.cuda_stream)
    if rc != COAT_OK:
        raise CoatError(rc, what)


def _workspace(nbytes: int, workspace: Optional[torch.Tensor], gpu: int, stream) -> Optional[torch.Tensor]:
    """The caller's workspace, or one of torch's allocator that lasts until the call's work is done."""
    if nbytes == 0:
        return None
    if workspace is not None:
        if workspace.get_device() != gpu or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous uint8 tensor on GPU {gpu}")
        if workspace.numel() < nbytes:
            raise ValueError(f"workspace has {workspace.numel()} bytes, the call needs {nbytes}")
        return workspace
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=gpu)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=gpu)


def mx4_code_bytes(k: int) -> int:
    """Code bytes of a row of k values in 4-bit form."""
    return (k + 127) // 128 * 64


def mx4_scale_bytes(k: int) -> int:
    """Scale bytes of a row of k values in 4-bit form."""
    return (k + 511) // 512 * 16


def mx4_empty(rows: int, k: int, device="cuda"):
    """Uninitialised (q, s) of a quantized matrix: rows of k values."""
    return (torch.empty(rows, mx4_code_bytes(k), dtype=torch.uint8, device=device),
            torch.empty(rows, mx4_scale_bytes(k), dtype=torch.uint8, device=device))


def _mx4_operand(q: torch.Tensor, s: torch.Tensor, rows: int, k: int, gpu: int, names=("q", "s")):
    return (_operand(q, torch.uint8, (rows, (k + 127) // 128 * 64), gpu, names[0]),
            _operand(s, torch.uint8, (rows, (k + 511) // 512 * 16), gpu, names[1]))


def mx4_quantize(x, q=None, s=None, q_t=None, s_t=None, *, stream=None) -> None:
    """A bf16 or fp32 matrix -> microscaled 4-bit codes and scale bytes, along its
    rows (q, s), its columns (q_t, s_t: the transposed matrix), or both in one pass."""
    gpu, ld, kind = _gpu_of(x, "x"), _row_stride(x, "x"), _float_type(x, "x")
    rows, cols = x.shape
    if (q is None) != (s is None) or (q_t is None) != (s_t is None) or (q is None and q_t is None):
        raise ValueError("codes and scales come in pairs: q with s, q_t with s_t, one pair at least")
    along = (None, None) if q is None else _mx4_operand(q, s, rows, cols, gpu)
    down = (None, None) if q_t is None else _mx4_operand(q_t, s_t, cols, rows, gpu, ("q_t", "s_t"))
    _call(gpu, stream, lib().coat_mx4_quantize, "coat_mx4_quantize", x.data_ptr(), rows, cols, ld, kind, *along, *down)


def mx4_dequantize(q, s, x, *, stream=None) -> None:
    """Microscaled 4-bit codes and scale bytes -> a bf16 or fp32 matrix."""
    gpu, ld, kind = _gpu_of(x, "x"), _row_stride(x, "x"), _float_type(x, "x")
    rows, cols = x.shape
    qp, sp = _mx4_operand(q, s, rows, cols, gpu)
    _call(gpu, stream, lib().coat_mx4_dequantize, "coat_mx4_dequantize", qp, sp, rows, cols, x.data_ptr(), ld, kind)


def mx4_matmul(a_q, a_s, b_q, b_s, y, *, workspace=None, stream=None) -> None:
    """y (m, n) = A B^T of two quantized matrices, A m x k and B n x k; y bf16 or fp32.

    k is taken from the codes, rounded up to 128 as they are. ``workspace``: uint8,
    at least ``mx4_matmul_workspace_bytes`` long; without one the call takes one
    from torch's allocator."""
    gpu, ld, kind = _gpu_of(y, "y"), _row_stride(y, "y"), _float_type(y, "y")
    m, n = y.shape
    if a_q.dim() != 2:
        raise ValueError("a_q must be a matrix")
    k = a_q.shape[1] * 2
    ap, asp = _mx4_operand(a_q, a_s, m, k, gpu, ("a_q", "a_s"))
    bp, bsp = _mx4_operand(b_q, b_s, n, k, gpu, ("b_q", "b_s"))
    L = lib()
    nbytes = L.coat_mx4_matmul_workspace_bytes(m, n, k)
    ws = _workspace(nbytes, workspace, gpu, stream)
    _call(gpu, stream, L.coat_mx4_matmul, "coat_mx4_matmul", ap, asp, m, bp, bsp, n, k, y.data_ptr(), ld, kind,
          ws.data_ptr() if ws is not None else None, nbytes)


def mx4_matmul_workspace_bytes(m: int, n: int, k: int) -> int:
    return lib().coat_mx4_matmul_workspace_bytes(m, n, k)


def _border(ref, w_post, w_pre, gate, rows_per_gate, scale, eps, post, res_type):
    """The border's description, its parameters' type and the gate's shape."""
    rows, cols = ref.shape
    dtype = None
    for t in (w_post, w_pre, gate):
        if t is not None:
            if dtype is not None and t.dtype is not dtype:
                raise ValueError(f"w_post, w_pre and gate must have one type, got {dtype} and {t.dtype}")
            dtype = t.dtype
    kind = 0
    if dtype is not None:
        kind = _TYPES.get(dtype)
        if kind is None:
            raise ValueError(f"w_post, w_pre and gate must be bfloat16 or float32, got {dtype}")
    if rows_per_gate is None:
        rows_per_gate = rows
    rpg = max(1, int(rows_per_gate)) if rows == 0 else int(rows_per_gate)
    if rpg < 1:
        raise ValueError("rows_per_gate must be at least 1")
    rpg = min(rpg, max(1, rows))  # more is the same, and may pass the 64 bits of the C call
    gates = (rows + rpg - 1) // rpg
    return _Border(rows, cols, rpg, eps, scale, 1 if post else 0, res_type, kind, 0), dtype, (gates, cols)


def block_norm(y, r, r_out=None, h=None, *, w_post=None, w_pre=None, gate=None, rows_per_gate=None, scale=1.0,
               eps=1e-5, post=None, q=None, q_scale=None, group: int = 0, fmt: int = 0, stream=None) -> None:
    """The border between two blocks: r_out = r + scale gate (w_post N(y)), h = w_pre N(r_out),
    N(a) = a / sqrt(mean(a^2) + eps) over the channels, eps at least 2^-126.

    y None: no addition, r itself is normalised. post: whether y is normalised
    (default: if w_post is given). gate: (ceil(rows / rows_per_gate), channels), token
    t takes row t // rows_per_gate (default: one row for all). The layer input goes to
    h (bf16) and/or to q, q_scale in a stored form: FP8 codes and fp32 scales as
    ``act_quantize`` writes them for the bf16 h (group 16 .. 512, dividing the
    channels), or with fmt FMT_MX4 as ``mx4_quantize`` does along the rows."""
    if r.dim() != 2:
        raise ValueError("r must be a matrix, one row per token")
    if post is None:
        post = w_post is not None
    shape = r.shape
    rows, cols = shape
    b, pt, gate_shape = _border(r, w_post, w_pre, gate, rows_per_gate, scale, eps, post, _float_type(r, "r"))
    bf16 = torch.bfloat16
    if q_scale is None and q is not None or q is None and q_scale is not None:
        raise ValueError("q and q_scale come as a pair")
    if q is not None and fmt not in (FMT_E4M3, FMT_E5M2, FMT_MX4):  # the C call would see the low 32 bits alone
        raise ValueError(f"fmt must be FMT_E4M3, FMT_E5M2 or FMT_MX4, got {fmt}")
    if q is not None and fmt != FMT_MX4 and (group < 1 or cols % group):
        raise ValueError(f"group {group} must divide the {cols} channels")
    gpu = _gpu_of(r, "r")
    qp = sp = None
    if q is not None:
        if fmt == FMT_MX4:
            group = 32
            qp, sp = _mx4_operand(q, q_scale, rows, cols, gpu, ("q", "q_scale"))
        else:
            qp = _operand(q, torch.uint8, shape, gpu, "q")
            sp = _operand(q_scale, torch.float32, (rows, cols // group), gpu, "q_scale")
    args = (_operand(y, bf16, shape, gpu, "y") if y is not None else None,
            _operand(r, r.dtype, shape, gpu, "r"),
            _operand(w_post, pt, (cols,), gpu, "w_post") if w_post is not None else None,
            _operand(w_pre, pt, (cols,), gpu, "w_pre") if w_pre is not None else None,
            _operand(gate, pt, gate_shape, gpu, "gate") if gate is not None else None,
            _operand(r_out, r.dtype, shape, gpu, "r_out") if r_out is not None else None,
            _operand(h, bf16, shape, gpu, "h") if h is not None else None)
    _call(gpu, stream, lib().coat_block_norm, "coat_block_norm", ctypes.byref(b), *args, qp, sp, group, fmt)


def block_norm_backward(y, r_out, dr_out, dh, dr, dy=None, *, w_post=None, w_pre=None, gate=None, rows_per_gate=None,
                        scale=1.0, eps=1e-5, post=None, dw_post=None, dw_pre=None, dgate=None, workspace=None,
                        stream=None) -> None:
    """Backward of ``block_norm`` from the stored r_out (r, if y was None): the gradients
    dr_out of r_out (None: zero) and dh of h (None: no norm before the next block) to dr
    and dy, and to dw_post, dw_pre and dgate where they are given (all bf16 or all
    fp32). ``workspace``: uint8, at least ``block_norm_backward_workspace_bytes`` long;
    without one the call takes one from torch's allocator."""
    if dr.dim() != 2:
        raise ValueError("dr must be a matrix, one row per token")
    if post is None:
        post = w_post is not None
    shape = dr.shape
    rows, cols = shape
    b, pt, gate_shape = _border(dr, w_post, w_pre, gate, rows_per_gate, scale, eps, post, _float_type(dr, "dr"))
    gt = None
    for t in (dw_post, dw_pre, dgate):
        if t is not None:
            if gt is not None and t.dtype is not gt:
                raise ValueError(f"dw_post, dw_pre and dgate must have one type, got {gt} and {t.dtype}")
            gt = t.dtype
            b.grad_type = _float_type(t, "a weight's gradient")
    gpu = _gpu_of(dr, "dr")
    bf16 = torch.bfloat16
    args = (_operand(y, bf16, shape, gpu, "y") if y is not None else None,
            _operand(r_out, dr.dtype, shape, gpu, "r_out") if r_out is not None else None,
            _operand(dr_out, dr.dtype, shape, gpu, "dr_out") if dr_out is not None else None,
            _operand(dh, bf16, shape, gpu, "dh") if dh is not None else None,
            _operand(w_post, pt, (cols,), gpu, "w_post") if w_post is not None else None,
            _operand(w_pre, pt, (cols,), gpu, "w_pre") if w_pre is not None else None,
            _operand(gate, pt, gate_shape, gpu, "gate") if gate is not None else None,
            _operand(dr, dr.dtype, shape, gpu, "dr"),
            _operand(dy, bf16, shape, gpu, "dy") if dy is not None else None,
            _operand(dw_post, gt, (cols,), gpu, "dw_post") if dw_post is not None else None,
            _operand(dw_pre, gt, (cols,), gpu, "dw_pre") if dw_pre is not None else None,
            _operand(dgate, gt, gate_shape, gpu, "dgate") if dgate is not None else None)
    nbytes = lib().coat_block_norm_backward_workspace_bytes(ctypes.byref(b)) if gt is not None else 0
    ws = _workspace(nbytes, workspace, gpu, stream)
    _call(gpu, stream, lib().coat_block_norm_backward, "coat_block_norm_backward", ctypes.byref(b), *args,
          ws.data_ptr() if ws is not None else None, nbytes)


def block_norm_backward_workspace_bytes(rows: int, cols: int, rows_per_gate: Optional[int] = None) -> int:
    rpg = rows if rows_per_gate is None else min(rows, rows_per_gate)
    b = _Border(rows, cols, max(1, rpg), 1e-5, 1.0, 0, 0, 0, 0)
    return lib().coat_block_norm_backward_workspace_bytes(ctypes.byref(b))


# ---------------------------------------------------------------- parameter lists

def _pad16(n: int) -> int:
    return (n + 15) // 16 * 16


@dataclass
class TensorState:
    """Views of one tensor's slice of the flat buffers of a ``ParamListState``."""
    params: torch.Tensor
    params_bf16: torch.Tensor
    grads: torch.Tensor
    m_q: torch.Tensor
    m_s: torch.Tensor
    m_k: torch.Tensor
    v_q: torch.Tensor
    v_s: torch.Tensor
    v_k: torch.Tensor


class ParamListState:
    """Flat device buffers for a whole parameter list and its FP8 Adam state.

    Each tensor's slice of every element buffer starts on a 16-element
    boundary (16-byte aligned FP8 codes); per-group arrays are packed.
    """

    def __init__(self, sizes: Sequence[int], group: int, device="cuda", with_bf16: bool = True):
        self.sizes = [int(n) for n in sizes]
        self.group = group
        self.offsets, self.goffsets = [], []
        off = goff = 0
        for n in self.sizes:
            self.offsets.append(off)
            self.goffsets.append(goff)
            off += _pad16(n)
            goff += ngroups(n, group)
        self.n_padded, self.n_groups = off, goff
        dev = torch.device(device)
        self.params = torch.zeros(off, dtype=torch.float32, device=dev)
        self.params_bf16 = torch.zeros(off, dtype=torch.bfloat16, device=dev) if with_bf16 else None
        self.grads = torch.zeros(off, dtype=torch.bfloat16, device=dev)
        self.m_q = torch.zeros(off, dtype=torch.uint8, device=dev)
        self.v_q = torch.zeros(off, dtype=torch.uint8, device=dev)
        self.m_s = torch.zeros(goff, dtype=torch.float64, device=dev)
        self.v_s = torch.zeros(goff, dtype=torch.float64, device=dev)
        self.m_k = torch.ones(goff, dtype=torch.float32, device=dev)
        self.v_k = torch.ones(goff, dtype=torch.float32, device=dev)
        self._plan = None
        self._workspace = None

    @property
    def n_params(self) -> int:
        return sum(self.sizes)

    def tensor(self, i: int) -> TensorState:
        o, n, go, ng = self.offsets[i], self.sizes[i], self.goffsets[i], ngroups(self.sizes[i], self.group)
        w = self.params_bf16[o:o + n] if self.params_bf16 is not None else None
        return TensorState(self.params[o:o + n], w, self.grads[o:o + n],
                           self.m_q[o:o + n], self.m_s[go:go + ng], self.m_k[go:go + ng],
                           self.v_q[o:o + n], self.v_s[go:go + ng], self.v_k[go:go + ng])

    def descriptors(self):
        arr = (_Tensor * len(self.sizes))()
        for i, n in enumerate(self.sizes):
            t = self.tensor(i)
            arr[i] = _Tensor(t.params.data_ptr(), t.params_bf16.data_ptr() if t.params_bf16 is not None else None,
                             t.grads.data_ptr(), t.m_q.data_ptr(), t.m_s.data_ptr(), t.m_k.data_ptr(),
                             t.v_q.data_ptr(), t.v_s.data_ptr(), t.v_k.data_ptr(), n)
        return arr

    def plan(self, stream=None) -> _Plan:
        """Upload the descriptor table once; reused by every ``step``."""
        if self._plan is None:
            L = lib()
            count = len(self.sizes)
            nbytes = L.coat_multi_workspace_bytes(count)
            self._workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.params.device)
            plan = _Plan()
            descs = self.descriptors()
            _check(L.coat_multi_plan_init(ctypes.byref(plan), descs, count, self._workspace.data_ptr(),
                                          nbytes, _stream(stream)), "coat_multi_plan_init")
            self._plan = plan
        return self._plan

    def step(self, *, fmt_m: int, fmt_v: int, lr: float, beta1: float, beta2: float, eps: float,
             weight_decay: float, step: int, stream=None) -> None:
        """One FP8-state AdamW step over every tensor, one kernel launch (asynchronous)."""
        plan = self.plan(stream)
        rc = lib().coat_fp8_adamw_step_planned(ctypes.byref(plan), self.group, fmt_m, fmt_v, lr, beta1,
                                               beta2, eps, weight_decay, step, _stream(stream))
        _check(rc, "coat_fp8_adamw_step_planned")

    def step_unplanned(self, *, fmt_m: int, fmt_v: int, lr: float, beta1: float, beta2: float,
                       eps: float, weight_decay: float, step: int, stream=None) -> None:
        """The same step through the one-call entry point (uploads the table each time)."""
        L = lib()
        count = len(self.sizes)
        nbytes = L.coat_multi_workspace_bytes(count)
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.params.device)
        rc = L.coat_fp8_adamw_step_multi(self.descriptors(), count, self.group, fmt_m, fmt_v, lr, beta1,
                                         beta2, eps, weight_decay, step, ws.data_ptr(), nbytes,
                                         _stream(stream))
        _check(rc, "coat_fp8_adamw_step_multi")
        # keep the workspace alive until the launch has run
        torch.cuda.current_stream().synchronize() if stream is None else stream.synchronize()

    def step_static(self, *, fmt_m: int, fmt_v: int, lr: float, beta1: float, beta2: float,
                    eps: float, weight_decay: float, step: int, stream=None) -> None:
        """The same step through the entry point that allocates nothing and
        keeps its tables in the library's own device array (asynchronous)."""
        rc = lib().coat_fp8_adamw_step_multi_static(self.descriptors(), len(self.sizes), self.group, fmt_m,
                                                     fmt_v, lr, beta1, beta2, eps, weight_decay, step,
                                                     _stream(stream))
        _check(rc, "coat_fp8_adamw_step_multi_static")

    # ------------------------------------------------------------ checkpoint
    #
    # The complete optimizer state is the fp32 master weights and the FP8
    # moments with their per-group scales and exponents (plus the step count,
    # which the caller owns). Grads are transient and the bf16 copy is the RNE
    # of the masters, so neither is saved. Stored compressed, as the kernels
    # keep it: 4 + 2 + 24/G bytes per parameter (6.19 at G = 128) against 12
    # for fp32 moments. A resumed run continues bit for bit.

    STATE_FIELDS = ("params", "m_q", "m_s", "m_k", "v_q", "v_s", "v_k")
    CHECKPOINT_FORMAT = "coat-fp8-adamw-state/1"

    def state_dict(self) -> Dict[str, torch.Tensor]:
        """The optimizer state as host tensors (copies of the flat buffers,
        per-tensor padding included). Waits for pending work on the current
        stream."""
        return {name: getattr(self, name).detach().to("cpu", copy=True) for name in self.STATE_FIELDS}

    def load_state_dict(self, sd: Dict[str, torch.Tensor]) -> None:
        """Copy a ``state_dict`` of a list with the same sizes and group size
        into the buffers (the plan stays valid: the buffers do not move)."""
        for name in self.STATE_FIELDS:
            dst = getattr(self, name)
            src = sd[name]
            if src.dtype != dst.dtype or src.shape != dst.shape:
                raise ValueError(f"checkpoint field {name}: {src.dtype} {tuple(src.shape)}, "
                                 f"expected {dst.dtype} {tuple(dst.shape)}")
            dst.copy_(src)

    def save(self, path: str, *, step: int, fmt_m: int, fmt_v: int) -> None:
        """Write the state to a safetensors file; `step` is the last step taken."""
        from safetensors.torch import save_file
        meta = {"format": self.CHECKPOINT_FORMAT, "sizes": json.dumps(self.sizes), "group": str(self.group),
                "step": str(int(step)), "fmt_m": str(int(fmt_m)), "fmt_v": str(int(fmt_v))}
        save_file(self.state_dict(), path, metadata=meta)

    @classmethod
    def load(cls, path: str, device="cuda", with_bf16: bool = True):
        """Rebuild a state from a file written by ``save``. Returns the state
        and the metadata (step, fmt_m, fmt_v as ints). The bf16 copy is not
        stored: it is written again by the next step."""
        from safetensors import safe_open
        with safe_open(path, framework="pt", device="cpu") as f:
            meta = f.metadata() or {}
            if meta.get("format") != cls.CHECKPOINT_FORMAT:
                raise ValueError(f"{path}: not a {cls.CHECKPOINT_FORMAT} checkpoint")
            st = cls(json.loads(meta["sizes"]), int(meta["group"]), device=device, with_bf16=with_bf16)
            st.load_state_dict({name: f.get_tensor(name) for name in cls.STATE_FIELDS})
        return st, {k: int(meta[k]) for k in ("step", "fmt_m", "fmt_v")}

    def quantize_moments(self, m: List[torch.Tensor], v: List[torch.Tensor], *, fmt_m: int, fmt_v: int,
                         stream=None) -> None:
        """Fill the FP8 state from fp32 moments, tensor by tensor."""
        for i in range(len(self.sizes)):
            t = self.tensor(i)
            quantize(m[i], t.m_q, t.m_s, t.m_k, group=self.group, fmt=fmt_m, stream=stream)
            quantize(v[i], t.v_q, t.v_s, t.v_k, group=self.group, fmt=fmt_v, stream=stream)
