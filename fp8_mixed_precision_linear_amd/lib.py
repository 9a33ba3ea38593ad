"""Thin Python binding of libfp8lin (the C ABI in include/fp8lin.h).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  Tensors are torch tensors on the GPU (PyTorch provides device
memory and streams); each call passes their device pointers and sizes to the
C function of the same name and raises Fp8Error on a non-OK status.  There
is no fallback: if libfp8lin.so is missing or fails to load, importing this
module raises.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8lin.so")

E4M3, E5M2 = 0, 1
SCALE_TENSOR, SCALE_1x128, SCALE_128x128 = 0, 1, 2
SCALE_1x128_POW2, SCALE_128x128_POW2 = 3, 4
SCALE_ROW = 5
OUT_BF16, OUT_F32, OUT_E4M3, OUT_E5M2 = 0, 1, 2, 3
AMAX_MAX, AMAX_MOST_RECENT = 0, 1
DT_BF16, DT_F32 = 0, 1
NORM_RMS, NORM_LAYER = 0, 1
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3
GATE_LINEAR, GATE_SIGMOID, GATE_TANH = 0, 1, 2
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = 0, 1, 2, 3, 4
EP_FEW_ROWS, EP_TILES, EP_LARGE = 0, 1, 2
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_BASE, ROPE_PARTS = 0, 1, 2, 3

STATUS = {0: "FP8_OK", 1: "FP8_ERR_NULL", 2: "FP8_ERR_SHAPE", 3: "FP8_ERR_ALIGN",
          4: "FP8_ERR_UNSUPPORTED", 5: "FP8_ERR_LAUNCH", 6: "FP8_ERR_ARG"}


class Fp8Error(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({text})")
        self.status = status


class GemmArgs(C.Structure):
    _fields_ = [("M", C.c_int64), ("N", C.c_int64), ("K", C.c_int64),
                ("lda", C.c_int64), ("ldb", C.c_int64), ("ldd", C.c_int64),
                ("A", C.c_void_p), ("a_fmt", C.c_int), ("a_scaling", C.c_int),
                ("a_scale_inv", C.c_void_p),
                ("B", C.c_void_p), ("b_fmt", C.c_int), ("b_scaling", C.c_int),
                ("b_scale_inv", C.c_void_p),
                ("D", C.c_void_p), ("d_dtype", C.c_int), ("d_amax", C.c_void_p),
                ("accumulate", C.c_int),
                ("d_scale", C.c_void_p), ("D_t", C.c_void_p), ("ldt", C.c_int64),
                ("amax_accumulate", C.c_int)]


class NormArgs(C.Structure):
    _fields_ = [("rows", C.c_int64), ("cols", C.c_int64),
                ("kind", C.c_int), ("stream_dtype", C.c_int), ("param_dtype", C.c_int),
                ("eps", C.c_float), ("res_scale", C.c_float), ("branch_scale", C.c_float),
                ("x", C.c_void_p), ("ldx", C.c_int64), ("z", C.c_void_p), ("ldz", C.c_int64),
                ("w_post", C.c_void_p), ("b_post", C.c_void_p), ("w_pre", C.c_void_p), ("b_pre", C.c_void_p),
                ("gate", C.c_void_p), ("ldg", C.c_int64), ("gate_kind", C.c_int), ("gate_act", C.c_int),
                ("h", C.c_void_p), ("ldh", C.c_int64), ("stats_z", C.c_void_p), ("stats_h", C.c_void_p),
                ("y", C.c_void_p), ("ldy", C.c_int64), ("y8", C.c_void_p), ("ldy8", C.c_int64),
                ("y8_format", C.c_int), ("y8_scaling", C.c_int),
                ("y8_scale", C.c_void_p), ("y8_scale_inv", C.c_void_p), ("y8_amax", C.c_void_p)]


class NormBwdArgs(C.Structure):
    _fields_ = [("rows", C.c_int64), ("cols", C.c_int64),
                ("kind", C.c_int), ("stream_dtype", C.c_int), ("param_dtype", C.c_int),
                ("res_scale", C.c_float), ("branch_scale", C.c_float),
                ("dy", C.c_void_p), ("lddy", C.c_int64), ("dh", C.c_void_p), ("lddh", C.c_int64),
                ("h", C.c_void_p), ("ldh", C.c_int64), ("stats_h", C.c_void_p),
                ("z", C.c_void_p), ("ldz", C.c_int64), ("stats_z", C.c_void_p),
                ("w_post", C.c_void_p), ("b_post", C.c_void_p), ("w_pre", C.c_void_p),
                ("gate", C.c_void_p), ("ldg", C.c_int64), ("gate_kind", C.c_int), ("gate_act", C.c_int),
                ("dx", C.c_void_p), ("lddx", C.c_int64), ("dz", C.c_void_p), ("lddz", C.c_int64),
                ("dgate", C.c_void_p), ("lddg", C.c_int64),
                ("dw_pre", C.c_void_p), ("db_pre", C.c_void_p), ("dw_post", C.c_void_p), ("db_post", C.c_void_p),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_int64)]


class EpilogueArgs(C.Structure):
    _fields_ = [("backward", C.c_int), ("act", C.c_int), ("param_dtype", C.c_int),
                ("bias", C.c_void_p), ("residual", C.c_void_p), ("ldres", C.c_int64),
                ("residual_dtype", C.c_int), ("res_scale", C.c_float),
                ("aux", C.c_void_p), ("ldaux", C.c_int64), ("dbias", C.c_void_p),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_int64)]


class EpPlan(C.Structure):
    _fields_ = [("kernel", C.c_int), ("tile_rows", C.c_int), ("k_parts", C.c_int)]


class GatedArgs(C.Structure):
    _fields_ = [("backward", C.c_int), ("act", C.c_int), ("param_dtype", C.c_int), ("bias", C.c_void_p),
                ("aux", C.c_void_p), ("ldaux", C.c_int64), ("ck", C.c_void_p), ("ldck", C.c_int64),
                ("ck_exp", C.c_void_p), ("ldexp", C.c_int64), ("dbias", C.c_void_p),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_int64)]


class RopeArgs(C.Structure):
    _fields_ = [("tokens", C.c_int64), ("q_heads", C.c_int64), ("k_heads", C.c_int64),
                ("dim", C.c_int64), ("pairs", C.c_int64),
                ("dtype", C.c_int), ("layout", C.c_int), ("inverse", C.c_int), ("scale", C.c_float),
                ("freqs", C.c_void_p), ("positions", C.c_void_p), ("positions_i64", C.c_int),
                ("offset", C.c_int64),
                ("q", C.c_void_p), ("q_token_stride", C.c_int64), ("q_head_stride", C.c_int64),
                ("k", C.c_void_p), ("k_token_stride", C.c_int64), ("k_head_stride", C.c_int64),
                ("q_out", C.c_void_p), ("q_out_token_stride", C.c_int64), ("q_out_head_stride", C.c_int64),
                ("k_out", C.c_void_p), ("k_out_token_stride", C.c_int64), ("k_out_head_stride", C.c_int64)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built: run `python -m fp8_mixed_precision_linear_amd.build`")
    L = C.CDLL(LIB_PATH)
    vp, i64, i32 = C.c_void_p, C.c_int64, C.c_int
    sig = {
        "fp8_abi_version": (i32, []),
        "fp8_status_string": (C.c_char_p, [i32]),
        "fp8_amax": (i32, [vp, i64, i64, i64, vp, vp]),
        "fp8_amax_acc": (i32, [vp, i64, i64, i64, vp, vp]),
        "fp8_cast_stats": (i32, [vp, i64, i64, i32, vp, vp, vp]),
        "fp8_compute_scale": (i32, [vp, i64, i32, i32, vp, vp, vp]),
        "fp8_compute_scale_pow2": (i32, [vp, i64, i32, i32, vp, vp, vp]),
        "fp8_amax_history_update": (i32, [vp, i64, i64, vp, i32, i32, i32, vp, vp, vp]),
        "fp8_amax_history_update_pow2": (i32, [vp, i64, i64, vp, i32, i32, i32, vp, vp, vp]),
        "fp8_amax_history_update_reset": (i32, [vp, i64, i64, vp, i32, i32, i32, vp, vp, vp]),
        "fp8_cast_amax_acc": (i32, [vp, i64, i64, i32, vp, vp, vp, vp, vp]),
        "fp8_cast_e4m3": (i32, [vp, i64, i64, vp, vp, vp, vp, vp]),
        "fp8_cast_e5m2": (i32, [vp, i64, i64, vp, vp, vp, vp, vp]),
        "fp8_cast_block": (i32, [vp, i64, i64, i32, i32, vp, vp, vp, vp, vp]),
        "fp8_cast_block_pow2": (i32, [vp, i64, i64, i32, i32, vp, vp, vp, vp, vp]),
        "fp8_cast_rowwise": (i32, [vp, i64, i64, i32, vp, vp, vp, vp, vp]),
        "fp8_cast_sr": (i32, [vp, i64, i64, i32, vp, C.c_uint64, C.c_uint64, vp, vp, vp, vp]),
        "fp8_cast_sr_state": (i32, [vp, i64, i64, i32, vp, vp, C.c_uint64, vp, vp, vp, vp]),
        "fp8_amax_ewma_update": (i32, [vp, i64, vp, C.c_float, i32, i32, vp, vp, vp]),
        "fp8_scaled_gemm": (i32, [C.POINTER(GemmArgs), vp]),
        "fp8_block_norm": (i32, [vp, vp]),
        "fp8_block_norm_bwd_workspace": (i64, [i64, i64]),
        "fp8_block_norm_bwd": (i32, [vp, vp]),
        "fp8_scaled_gemm_ep_workspace": (i64, [i64, i64, i64, i32, i32]),
        "fp8_scaled_gemm_ep": (i32, [vp, vp, vp]),
        "fp8_scaled_gemm_ep_plan": (i32, [vp, vp, vp]),
        "fp8_gated_linear_workspace": (i64, [i64, i64, i64, i32, i32, i32]),
        "fp8_gated_linear": (i32, [vp, vp, vp]),
        "fp8_gated_linear_plan": (i32, [vp, vp, vp]),
        "fp8_checkpoint_save": (i32, [vp, i32, i64, i64, i64, vp, i64, vp, i64, vp]),
        "fp8_checkpoint_load": (i32, [vp, i64, vp, i64, i64, i64, vp, i32, i64, vp]),
        "fp8_rope": (i32, [vp, vp]),
        "fp8_rope_freqs": (i32, [vp, i64, C.c_double, i32, C.c_double, C.c_double, C.c_double, C.c_double, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    return L


_L = _load()


def abi_version() -> int:
    return _L.fp8_abi_version()


def status_string(status: int) -> str:
    return _L.fp8_status_string(status).decode()


def _check(fn: str, status: int):
    if status != 0:
        raise Fp8Error(fn, status, status_string(status))


def _ptr(t, dtypes=None, name="tensor"):
    """Device pointer of a GPU tensor (None -> NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() or None


def _stream(stream):
    if stream is None:   # the handle of torch.cuda.current_stream(), without the object
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _stream_on(dev, stream):
    """_stream of a call whose tensors are on GPU dev: the current device, where the
    launch goes, and an explicit stream's."""
    here = torch._C._cuda_getDevice()
    if dev != here:
        raise ValueError(f"the operands are on cuda:{dev}, the current device is cuda:{here}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(here)
    if isinstance(stream, torch.cuda.Stream):
        if stream.device_index != here:
            raise ValueError(f"the stream is of cuda:{stream.device_index}, the operands are on cuda:{here}")
        return stream.cuda_stream
    return int(stream)


_BF16 = (torch.bfloat16,)
_F32 = (torch.float32,)
_I64 = (torch.int64,)
_U8 = (torch.uint8, torch.float8_e4m3fn, torch.float8_e5m2)
_POWERS = (torch.uint8, torch.float8_e8m0fnu)


def _need(t, n, name):
    """Raise unless tensor t (if given) holds at least n elements: the C ABI
    cannot see buffer sizes, so the binding checks them before any launch."""
    if t is not None and t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} elements, the call needs {n}")


def _rc(x):
    """(rows, cols) of a tensor viewed as [rows][cols] (1-D: one row)."""
    if x.dim() == 0:
        return 1, 1
    if x.dim() == 1:
        return 1, x.shape[0]
    cols = 1
    for d in x.shape[1:]:
        cols *= d
    return x.shape[0], cols


def _amax(fn, x, amax, stream):
    _need(amax, 1, "amax")
    if x.dim() == 2 and not x.is_contiguous() and x.stride(1) == 1 and x.stride(0) >= x.shape[1]:
        rows, cols, ld = x.shape[0], x.shape[1], x.stride(0)
        if not x.is_cuda or x.dtype not in _BF16:
            raise TypeError("x must be a bf16 GPU tensor")
        xp = x.data_ptr() or None
    else:
        rows, cols = _rc(x)
        ld = cols
        xp = _ptr(x, _BF16, "x")
    _check(fn.__name__, fn(xp, rows, cols, ld, _ptr(amax, _F32, "amax"), _stream(stream)))


def fp8_amax(x, amax, stream=None):
    """amax of x: a contiguous tensor, or a 2-D view whose rows are strided
    (row stride >= number of columns, unit column stride)."""
    _amax(_L.fp8_amax, x, amax, stream)


def fp8_cast_stats(x, fmt, scale, counts, stream=None):
    """Adds the cast's saturated / underflowed element counts of x (scale
    scale[0], format fmt) to counts[0] / counts[1] (an int64 tensor of 2)."""
    rows, cols = _rc(x)
    _need(scale, 1, "scale")
    if counts is None or counts.dtype != torch.int64 or counts.numel() < 2 or not counts.is_cuda:
        raise ValueError("counts must be a GPU int64 tensor of 2")
    _check("fp8_cast_stats",
           _L.fp8_cast_stats(_ptr(x, _BF16, "x"), rows, cols, fmt, _ptr(scale, _F32, "scale"),
                             counts.data_ptr(), _stream(stream)))


def fp8_amax_acc(x, amax_acc, stream=None):
    """fp8_amax max-accumulated into amax_acc (no fill ahead of the kernel)."""
    if amax_acc is None:
        raise ValueError("amax_acc is required")
    _amax(_L.fp8_amax_acc, x, amax_acc, stream)


def _compute_scale(fn, amax, fmt, margin, scale, scale_inv, stream):
    _need(scale, amax.numel(), "scale")
    _need(scale_inv, amax.numel(), "scale_inv")
    _check(fn.__name__,
           fn(_ptr(amax, _F32, "amax"), amax.numel(), fmt, margin,
              _ptr(scale, _F32, "scale"), _ptr(scale_inv, _F32, "scale_inv"), _stream(stream)))


def fp8_compute_scale(amax, fmt, margin, scale, scale_inv, stream=None):
    _compute_scale(_L.fp8_compute_scale, amax, fmt, margin, scale, scale_inv, stream)


def fp8_compute_scale_pow2(amax, fmt, margin, scale, scale_inv, stream=None):
    _compute_scale(_L.fp8_compute_scale_pow2, amax, fmt, margin, scale, scale_inv, stream)


def _history(fn, history, amax_new, fmt, margin, algo, scale, scale_inv, stream):
    n, ln = history.shape
    for name, t in (("amax_new", amax_new), ("scale", scale), ("scale_inv", scale_inv)):
        _need(t, n, name)
    _check(fn.__name__,
           fn(_ptr(history, _F32, "history"), n, ln, _ptr(amax_new, _F32, "amax_new"), fmt, margin,
              algo, _ptr(scale, _F32, "scale"), _ptr(scale_inv, _F32, "scale_inv"), _stream(stream)))


def fp8_amax_history_update(history, amax_new, fmt, margin, algo, scale, scale_inv, stream=None):
    _history(_L.fp8_amax_history_update, history, amax_new, fmt, margin, algo, scale, scale_inv,
             stream)


def fp8_amax_history_update_pow2(history, amax_new, fmt, margin, algo, scale, scale_inv,
                                 stream=None):
    _history(_L.fp8_amax_history_update_pow2, history, amax_new, fmt, margin, algo, scale,
             scale_inv, stream)


def fp8_amax_history_update_reset(history, amax_new, fmt, margin, algo, scale, scale_inv,
                                  stream=None):
    """fp8_amax_history_update, then amax_new is set to 0 (the slots the next
    step's fp8_cast_amax_acc calls accumulate into)."""
    _history(_L.fp8_amax_history_update_reset, history, amax_new, fmt, margin, algo, scale,
             scale_inv, stream)


def fp8_cast_amax_acc(x, fmt, scale, amax_acc, y=None, y_t=None, stream=None):
    """Per-tensor cast with the amax of x max-accumulated into amax_acc."""
    if amax_acc is None:
        raise ValueError("amax_acc is required")
    rows, cols = _cast_sizes(x, scale, y, y_t, amax_acc)
    _check("fp8_cast_amax_acc",
           _L.fp8_cast_amax_acc(_ptr(x, _BF16, "x"), rows, cols, fmt, _ptr(scale, _F32, "scale"),
                                _ptr(y, _U8, "y"), _ptr(y_t, _U8, "y_t"),
                                _ptr(amax_acc, _F32, "amax_acc"), _stream(stream)))


def _cast_sizes(x, scale, y, y_t, amax_out):
    rows, cols = _rc(x)
    _need(scale, 1, "scale")
    _need(y, rows * cols, "y")
    _need(y_t, rows * cols, "y_t")
    _need(amax_out, 1, "amax_out")
    return rows, cols


def _cast(fn, x, scale, y, y_t, amax_out, stream):
    rows, cols = _cast_sizes(x, scale, y, y_t, amax_out)
    _check(fn.__name__, fn(_ptr(x, _BF16, "x"), rows, cols, _ptr(scale, _F32, "scale"),
                           _ptr(y, _U8, "y"), _ptr(y_t, _U8, "y_t"),
                           _ptr(amax_out, _F32, "amax_out"), _stream(stream)))


def fp8_cast_sr(x, fmt, scale, seed, offset=0, y=None, y_t=None, amax_out=None, stream=None):
    rows, cols = _cast_sizes(x, scale, y, y_t, amax_out)
    _check("fp8_cast_sr",
           _L.fp8_cast_sr(_ptr(x, _BF16, "x"), rows, cols, fmt, _ptr(scale, _F32, "scale"),
                          int(seed), int(offset), _ptr(y, _U8, "y"), _ptr(y_t, _U8, "y_t"),
                          _ptr(amax_out, _F32, "amax_out"), _stream(stream)))


def fp8_cast_sr_state(x, fmt, scale, rng_state, advance=1, y=None, y_t=None, amax_out=None,
                      stream=None):
    """Stochastic-rounding cast whose (seed, offset) are read on the device
    from rng_state (an int64 tensor of 2: seed, offset, as unsigned 64-bit
    words); rng_state[1] then moves on by `advance` in stream order, so a
    replayed graph draws fresh words each time."""
    rows, cols = _cast_sizes(x, scale, y, y_t, amax_out)
    if rng_state.numel() < 2:
        raise ValueError("rng_state needs 2 elements (seed, offset)")
    _check("fp8_cast_sr_state",
           _L.fp8_cast_sr_state(_ptr(x, _BF16, "x"), rows, cols, fmt, _ptr(scale, _F32, "scale"),
                                _ptr(rng_state, _I64, "rng_state"), int(advance),
                                _ptr(y, _U8, "y"), _ptr(y_t, _U8, "y_t"),
                                _ptr(amax_out, _F32, "amax_out"), _stream(stream)))


def fp8_amax_ewma_update(ewma, amax_new, beta, fmt, margin, scale, scale_inv, stream=None):
    n = ewma.numel()
    for name, t in (("amax_new", amax_new), ("scale", scale), ("scale_inv", scale_inv)):
        if t.numel() != n:
            raise ValueError(f"{name} must hold {n} floats")
    _check("fp8_amax_ewma_update",
           _L.fp8_amax_ewma_update(_ptr(ewma, _F32, "ewma"), n, _ptr(amax_new, _F32, "amax_new"),
                                   float(beta), fmt, margin, _ptr(scale, _F32, "scale"),
                                   _ptr(scale_inv, _F32, "scale_inv"), _stream(stream)))


def fp8_cast_e4m3(x, scale, y=None, y_t=None, amax_out=None, stream=None):
    _cast(_L.fp8_cast_e4m3, x, scale, y, y_t, amax_out, stream)


def fp8_cast_e5m2(x, scale, y=None, y_t=None, amax_out=None, stream=None):
    _cast(_L.fp8_cast_e5m2, x, scale, y, y_t, amax_out, stream)


def _cast_block(fn, x, fmt, tile, y, scale_inv, y_t, scale_inv_t, stream):
    rows, cols = _rc(x)
    nrb, ncb = (rows + 127) // 128, (cols + 127) // 128
    _need(y, rows * cols, "y")
    _need(y_t, rows * cols, "y_t")
    _need(scale_inv, ncb * (rows if tile == SCALE_1x128 else nrb), "scale_inv")
    _need(scale_inv_t, nrb * (cols if tile == SCALE_1x128 else ncb), "scale_inv_t")
    _check(fn.__name__,
           fn(_ptr(x, _BF16, "x"), rows, cols, fmt, tile, _ptr(y, _U8, "y"),
              _ptr(scale_inv, _F32, "scale_inv"), _ptr(y_t, _U8, "y_t"),
              _ptr(scale_inv_t, _F32, "scale_inv_t"), _stream(stream)))


def fp8_cast_block(x, fmt, tile, y=None, scale_inv=None, y_t=None, scale_inv_t=None, stream=None):
    _cast_block(_L.fp8_cast_block, x, fmt, tile, y, scale_inv, y_t, scale_inv_t, stream)


def fp8_cast_block_pow2(x, fmt, tile, y=None, scale_inv=None, y_t=None, scale_inv_t=None,
                        stream=None):
    _cast_block(_L.fp8_cast_block_pow2, x, fmt, tile, y, scale_inv, y_t, scale_inv_t, stream)


def fp8_cast_rowwise(x, fmt, y=None, scale_inv=None, y_t=None, scale_inv_t=None, stream=None):
    rows, cols = _rc(x)
    _need(y, rows * cols, "y")
    _need(scale_inv, rows, "scale_inv")
    _need(y_t, rows * cols, "y_t")
    _need(scale_inv_t, cols, "scale_inv_t")
    _check("fp8_cast_rowwise",
           _L.fp8_cast_rowwise(_ptr(x, _BF16, "x"), rows, cols, fmt, _ptr(y, _U8, "y"),
                               _ptr(scale_inv, _F32, "scale_inv"), _ptr(y_t, _U8, "y_t"),
                               _ptr(scale_inv_t, _F32, "scale_inv_t"), _stream(stream)))


def fp8_scaled_gemm(A, a_fmt, a_scaling, a_scale_inv, B, b_fmt, b_scaling, b_scale_inv, D,
                    d_amax=None, accumulate=False, stream=None, d_scale=None, d_fmt=None, D_t=None,
                    amax_accumulate=False):
    """D [M][N] = A [M][K] . B [N][K]^T with FP8 codes.  D is a bf16 or fp32
    tensor, or a uint8 tensor of FP8 codes (d_fmt E4M3 / E5M2, quantised
    with d_scale; D_t optional [N][M] transposed codes).  d_amax receives
    max |output|, max-accumulated into its value with amax_accumulate."""
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K or tuple(D.shape) != (M, N):
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, D {tuple(D.shape)}")
    if D.dtype in _U8:
        if d_fmt not in (E4M3, E5M2):
            raise ValueError("an FP8 output needs d_fmt (E4M3 or E5M2)")
        d_dtype = OUT_E4M3 if d_fmt == E4M3 else OUT_E5M2
        if D_t is not None and tuple(D_t.shape) != (N, M):
            raise ValueError(f"D_t must be [{N}][{M}], got {tuple(D_t.shape)}")
    else:
        d_dtype = {torch.bfloat16: OUT_BF16, torch.float32: OUT_F32}[D.dtype]
    nkb = (K + 127) // 128

    def scales_needed(scaling, rows):
        if scaling in (SCALE_1x128, SCALE_1x128_POW2):
            return nkb * rows
        if scaling in (SCALE_128x128, SCALE_128x128_POW2):
            return nkb * ((rows + 127) // 128)
        return rows if scaling == SCALE_ROW else 1
    if K > 0 and M > 0 and N > 0:
        _need(a_scale_inv, scales_needed(a_scaling, M), "a_scale_inv")
        _need(b_scale_inv, scales_needed(b_scaling, N), "b_scale_inv")
    _need(d_amax, 1, "d_amax")
    _need(d_scale, 1, "d_scale")
    g = GemmArgs(M, N, K, K, K, N,
                 _ptr(A, _U8, "A"), a_fmt, a_scaling, _ptr(a_scale_inv, _F32, "a_scale_inv"),
                 _ptr(B, _U8, "B"), b_fmt, b_scaling, _ptr(b_scale_inv, _F32, "b_scale_inv"),
                 _ptr(D, None, "D"), d_dtype, _ptr(d_amax, _F32, "d_amax"), 1 if accumulate else 0,
                 _ptr(d_scale, _F32, "d_scale"), _ptr(D_t, _U8, "D_t"), M,
                 1 if amax_accumulate else 0)
    _check("fp8_scaled_gemm", _L.fp8_scaled_gemm(C.byref(g), _stream(stream)))


# ---------------------------------------------------------------------------
# Operators around the linears: norms with the block's gate and residual
# scale, the GEMM with the linear's epilogue, rotary positions.
#
# One token's call is over in less time than a Structure of 30 fields takes to
# fill, so the argument blocks are packed in one step (the layouts are checked
# against the Structures below) and each tensor is looked at once.

_DT = {torch.bfloat16: DT_BF16, torch.float32: DT_F32}
_BFLOAT, _FLOAT = torch.bfloat16, torch.float32


def _packer(fmt, structure):
    s = struct.Struct("@" + fmt + "0q")
    if s.size != C.sizeof(structure):
        raise ImportError(f"layout of {structure.__name__}: {s.size} bytes packed, {C.sizeof(structure)} declared")
    return s.pack


_pack_gemm = _packer("qqqqqqPiiPPiiPPiPiPPqi", GemmArgs)
_pack_norm = _packer("qqiiifffPqPqPPPPPqiiPqPPPqPqiiPPP", NormArgs)
_pack_norm_bwd = _packer("qqiiiffPqPqPqPPqPPPPPqiiPqPqPqPPPPPq", NormBwdArgs)
_pack_ep = _packer("iiiPPqifPqPPq", EpilogueArgs)
_pack_gated = _packer("iiiPPqPqPqPPq", GatedArgs)
_pack_rope = _packer("qqqqqiiifPPiqPqqPqqPqqPqq", RopeArgs)


def _refuse(t, want, dtype, name, dev=None):
    """What is wrong with a tensor that should have been [want] of dtype, on GPU dev."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a GPU tensor")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the call's first operand on cuda:{dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be {tuple(want)} with rows of unit stride that do not overlap, got "
                     f"{tuple(t.shape)}, strides {t.stride()}")


def _mat(t, shape, dtype, name, dev=None):
    """(pointer, row stride) of a 2-D GPU tensor of that shape and type, whose
    rows may be strided; (0, columns) for None.  dev: the GPU that it has to be on
    (None: any)."""
    if t is None:
        return 0, shape[1]
    if t.dtype != dtype or t.shape != shape or (not t.is_cuda if dev is None else not 0 <= dev == t.get_device()):
        _refuse(t, shape, dtype, name, dev)
    if t.is_contiguous():
        return t.data_ptr(), shape[1]
    ld, one = t.stride()
    if shape[0] == 1:
        ld = shape[1]
    if (one != 1 and shape[1] > 1) or ld < shape[1]:
        _refuse(t, shape, dtype, name)
    return t.data_ptr(), ld


def _codes(t, shape, name, dev=None):
    """_mat of FP8 codes (uint8 or a float8 type)."""
    if t is not None and t.dtype not in _U8:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {_U8}")
    return _mat(t, shape, None if t is None else t.dtype, name, dev)


def _vec(t, n, dtype, name, dev=None):
    """Pointer of a contiguous 1-D GPU tensor of n elements (None -> 0)."""
    if t is None:
        return 0
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or (not t.is_cuda if dev is None else not 0 <= dev == t.get_device()) or not t.is_contiguous():
        _refuse(t, (n,), dtype, name, dev)
    return t.data_ptr()


def _floats(t, n, name, dev=None):
    """Pointer of a contiguous float32 GPU tensor of at least n elements."""
    if t is None:
        return 0
    if t.dtype != _FLOAT or (not t.is_cuda if dev is None else not 0 <= dev == t.get_device()) or not t.is_contiguous():
        _refuse(t, (n,), _FLOAT, name, dev)
    if t.numel() < n:
        _need(t, n, name)
    return t.data_ptr()


def _param_type(*vectors):
    """The one type of a call's parameters, from the first that is given."""
    for t in vectors:
        if t is not None:
            if t.dtype not in _DT:
                raise TypeError(f"parameters must be bf16 or float32, got {t.dtype}")
            return t.dtype
    return _FLOAT


def _gate(gate, shape, ptype, name="gate"):
    """(kind, pointer, row stride) of a gate: [cols], [rows, 1] or [rows, cols]."""
    rows, cols = shape
    if gate is None:
        return GATE_NONE, 0, cols
    if gate.dim() == 1:
        return GATE_CHANNEL, _vec(gate, cols, ptype, name), cols
    if gate.dtype == _FLOAT:
        if gate.shape != (rows, 1) or not gate.is_cuda or not gate.is_contiguous():
            _refuse(gate, (rows, 1), _FLOAT, f"a float32 (per-token) {name}")
        return GATE_TOKEN, gate.data_ptr(), cols
    return (GATE_FULL, *_mat(gate, shape, _BFLOAT, name))


def _workspace(ws, need, like, stream, dev=None):
    """(tensor, pointer, bytes) of the caller's workspace, or of one from
    torch's allocator (on the current stream only, whose order keeps it)."""
    if ws is None:
        if stream is not None:
            raise ValueError("a call on an explicit stream needs a workspace")
        n = need()
        if n == 0:
            return None, 0, 0
        ws = torch.empty(n, dtype=torch.uint8, device=like.device)
    elif not ws.is_cuda or not ws.is_contiguous() or (dev is not None and ws.get_device() != dev):
        raise ValueError("workspace must be a contiguous GPU tensor, on the operands' device")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _two_dim(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(t.shape)}")
    if t.dtype not in _DT:
        raise TypeError(f"{name} must be bf16 or float32, got {t.dtype}")
    return t.shape


def fp8_block_norm(x, z=None, h=None, y=None, kind=NORM_RMS, eps=1e-6, w_pre=None, b_pre=None,
                   w_post=None, b_post=None, gate=None, gate_act=GATE_LINEAR, res_scale=1.0,
                   branch_scale=1.0, stats_z=None, stats_h=None, y8=None, y8_fmt=E4M3,
                   y8_scaling=SCALE_TENSOR, y8_scale=None, y8_scale_inv=None, y8_amax=None, stream=None):
    """h = res_scale * x + branch_scale * gate * N(z), y = N(h), row by row.

    x [rows][cols], bf16 or float32, is the residual stream, z [rows][cols]
    bf16 the output of the block that ends here (None: h is x), h the new
    stream (x's type; may be x).  y is bf16; y8 holds FP8 codes of y with
    y8_scaling SCALE_TENSOR (y8_scale given, y8_amax max-accumulated),
    SCALE_ROW or SCALE_1x128 (y8_scale_inv written), row by row (a transposed
    copy is fp8_cast_*'s).  Weights and biases [cols]
    and a per-channel gate [cols] share one type; a gate [rows, 1] is float32, a
    gate [rows, cols] bf16.  stats_z / stats_h [rows, 2] float32 receive (mean,
    1 / deviation) for fp8_block_norm_bwd."""
    shape = _two_dim(x, "x")
    rows, cols = shape
    st = x.dtype
    pt = _param_type(w_pre, w_post, b_pre, b_post, gate if gate is not None and gate.dim() == 1 else None)
    gk, gp, ldg = _gate(gate, shape, pt)
    nsi = 0 if y8_scaling == SCALE_TENSOR else rows if y8_scaling == SCALE_ROW else (cols + 127) // 128 * rows
    a = _pack_norm(rows, cols, kind, _DT[st], _DT[pt], eps, res_scale, branch_scale, *_mat(x, shape, st, "x"),
                   *_mat(z, shape, _BFLOAT, "z"), _vec(w_post, cols, pt, "w_post"), _vec(b_post, cols, pt, "b_post"),
                   _vec(w_pre, cols, pt, "w_pre"), _vec(b_pre, cols, pt, "b_pre"), gp, ldg, gk, gate_act,
                   *_mat(h, shape, st, "h"), _floats(stats_z, 2 * rows, "stats_z"),
                   _floats(stats_h, 2 * rows, "stats_h"), *_mat(y, shape, _BFLOAT, "y"), *_codes(y8, shape, "y8"),
                   y8_fmt, y8_scaling, _floats(y8_scale, 1, "y8_scale"), _floats(y8_scale_inv, nsi, "y8_scale_inv"),
                   _floats(y8_amax, 1, "y8_amax"))
    status = _L.fp8_block_norm(a, _stream(stream))
    if status:
        _check("fp8_block_norm", status)


def fp8_block_norm_bwd_workspace(rows, cols) -> int:
    """Bytes of workspace that fp8_block_norm_bwd needs."""
    return _L.fp8_block_norm_bwd_workspace(rows, cols)


def fp8_block_norm_bwd(h, dx, dy=None, dh=None, z=None, dz=None, kind=NORM_RMS, w_pre=None, w_post=None,
                       b_post=None, gate=None, gate_act=GATE_LINEAR, res_scale=1.0, branch_scale=1.0,
                       stats_z=None, stats_h=None, dw_pre=None, db_pre=None, dw_post=None, db_post=None,
                       dgate=None, workspace=None, stream=None):
    """Gradients of fp8_block_norm: of x (dx), z (dz), the weights, biases and
    the gate, from dy (of y; None: y was not made) and dh (what reaches h from
    above; None: nothing).  h, z and the statistics are the forward call's (h:
    x where there was no z).  Every output may be left out (dx too: None); dx
    may be dh and dz may be dy."""
    shape = _two_dim(h, "h")
    rows, cols = shape
    st = h.dtype
    pt = _param_type(w_pre, w_post, dw_pre, dw_post, b_post, db_pre, db_post,
                     gate if gate is not None and gate.dim() == 1 else None)
    gk, gp, ldg = _gate(gate, shape, pt)
    dgp, lddg = 0, cols
    if dgate is not None:
        if gate is None or dgate.shape != gate.shape or dgate.dtype != gate.dtype:
            raise ValueError("dgate must have the gate's shape and type")
        _, dgp, lddg = _gate(dgate, shape, pt, "dgate")
    ws, wp, wn = _workspace(workspace, lambda: _L.fp8_block_norm_bwd_workspace(rows, cols), h, stream)
    a = _pack_norm_bwd(rows, cols, kind, _DT[st], _DT[pt], res_scale, branch_scale, *_mat(dy, shape, _BFLOAT, "dy"),
                       *_mat(dh, shape, st, "dh"), *_mat(h, shape, st, "h"), _floats(stats_h, 2 * rows, "stats_h"),
                       *_mat(z, shape, _BFLOAT, "z"), _floats(stats_z, 2 * rows, "stats_z"),
                       _vec(w_post, cols, pt, "w_post"), _vec(b_post, cols, pt, "b_post"),
                       _vec(w_pre, cols, pt, "w_pre"), gp, ldg, gk, gate_act, *_mat(dx, shape, st, "dx"),
                       *_mat(dz, shape, _BFLOAT, "dz"), dgp, lddg, _vec(dw_pre, cols, pt, "dw_pre"),
                       _vec(db_pre, cols, pt, "db_pre"), _vec(dw_post, cols, pt, "dw_post"),
                       _vec(db_post, cols, pt, "db_post"), wp, wn)
    status = _L.fp8_block_norm_bwd(a, _stream(stream))
    if status:
        _check("fp8_block_norm_bwd", status)


def fp8_scaled_gemm_ep_workspace(M, N, K, a_scaling, b_scaling) -> int:
    """Bytes of workspace that fp8_scaled_gemm_ep needs."""
    return _L.fp8_scaled_gemm_ep_workspace(M, N, K, a_scaling, b_scaling)


def _scales(t, scaling, rows, nkb, name, dev=None):
    n = (1 if scaling == SCALE_TENSOR else rows if scaling == SCALE_ROW else
         nkb * (rows if scaling in (SCALE_1x128, SCALE_1x128_POW2) else (rows + 127) // 128))
    return _floats(t, n if nkb > 0 else 0, name, dev)


_OUT = {torch.bfloat16: OUT_BF16, torch.float32: OUT_F32}


def fp8_scaled_gemm_ep(A, a_fmt, a_scaling, a_scale_inv, B, b_fmt, b_scaling, b_scale_inv, D, bias=None,
                       act=ACT_NONE, aux=None, residual=None, res_scale=1.0, backward=False, dbias=None,
                       d_amax=None, stream=None, d_scale=None, d_fmt=None, D_t=None, amax_accumulate=False,
                       workspace=None):
    """fp8_scaled_gemm with the linear's epilogue.  With v the dequantised
    product: forward, u = v + bias, aux = bf16(u) if given, D = act(u) +
    res_scale * residual; backward, D = v * act'(aux) and dbias = column sums
    of it.  D is bf16, float32, or FP8 codes (uint8 or float8; d_fmt, d_scale,
    optional transposed D_t).  A, B, D, D_t, aux and residual may have strided
    rows; bias and dbias are [N] bf16 or float32."""
    M, K = A.shape
    N = B.shape[0]
    mn = torch.Size((M, N))
    dt = D.dtype
    if dt in _U8:
        if d_fmt not in (E4M3, E5M2):
            raise ValueError("an FP8 output needs d_fmt (E4M3 or E5M2)")
        d_dtype = OUT_E4M3 if d_fmt == E4M3 else OUT_E5M2
    elif dt in _OUT:
        d_dtype = _OUT[dt]
    else:
        raise TypeError(f"D has dtype {dt}, expected bf16, float32 or FP8 codes")
    pt = _param_type(bias, dbias)
    rt = _BFLOAT if residual is None else residual.dtype
    if rt not in _DT:
        raise TypeError(f"residual must be bf16 or float32, got {rt}")
    nkb = (K + 127) // 128 if M > 0 and N > 0 else 0
    ap, lda = _codes(A, A.shape, "A")
    bp, ldb = _codes(B, torch.Size((N, K)), "B")
    dp, ldd = _mat(D, mn, dt, "D")
    tp, ldt = _codes(D_t, torch.Size((N, M)), "D_t") if D_t is not None else (0, M)
    ws, wp, wn = _workspace(workspace, lambda: _L.fp8_scaled_gemm_ep_workspace(M, N, K, a_scaling, b_scaling), A,
                            stream)
    g = _pack_gemm(M, N, K, lda, ldb, ldd, ap, a_fmt, a_scaling, _scales(a_scale_inv, a_scaling, M, nkb, "a_scale_inv"),
                   bp, b_fmt, b_scaling, _scales(b_scale_inv, b_scaling, N, nkb, "b_scale_inv"), dp, d_dtype,
                   _floats(d_amax, 1, "d_amax"), 0, _floats(d_scale, 1, "d_scale"), tp, ldt,
                   1 if amax_accumulate else 0)
    e = _pack_ep(1 if backward else 0, act, _DT[pt], _vec(bias, N, pt, "bias"), *_mat(residual, mn, rt, "residual"),
                 _DT[rt], res_scale, *_mat(aux, mn, _BFLOAT, "aux"), _vec(dbias, N, pt, "dbias"), wp, wn)
    status = _L.fp8_scaled_gemm_ep(g, e, _stream(stream))
    if status:
        _check("fp8_scaled_gemm_ep", status)


def fp8_gated_linear_workspace(M, F, K, a_scaling, b_scaling, backward=False) -> int:
    """Bytes of workspace that fp8_gated_linear needs."""
    return _L.fp8_gated_linear_workspace(M, F, K, a_scaling, b_scaling, 1 if backward else 0)


def fp8_gated_linear(A, a_fmt, a_scaling, a_scale_inv, B, b_fmt, b_scaling, b_scale_inv, D, act=ACT_SILU, bias=None,
                     aux=None, ck=None, ck_exp=None, backward=False, dbias=None, d_amax=None, stream=None, d_scale=None,
                     d_fmt=None, D_t=None, amax_accumulate=False, workspace=None):
    """The gated pair of a feed-forward block as one FP8 product.

    Forward: A [M][K], B [2F][K] (the gate's rows, then the up projection's); g, u
    = halves of A B^T + bias [2F]; D [M][F] = act(g) * u.  Backward: A [M][K] the
    gradient of the next linear's output, B [F][K] that linear's weights; v = A B^T;
    D [M][2F] = (v * u * act'(g) | v * act(g)), dbias [2F] its column sums.  D is
    bf16, float32, or FP8 codes (uint8 or float8; d_fmt, d_scale, optional
    transposed D_t).  g beside u are kept by the forward call, and read by the
    backward one, as aux [M][2F] bf16 or as ck [M][2F] codes with ck_exp
    [M][2 ceil(F / 32)] (see fp8_checkpoint_save).  All but the scales and biases may
    have strided rows.  Large calls are fastest where every row of D, D_t, aux and ck
    starts on a multiple of 4 bytes: with M no multiple of 4, where D_t is a view of
    rows padded to one (1.4 times faster than a contiguous D_t; a product over the
    tokens takes it with zeros up to a multiple of 16).  Every tensor is on the current
    device."""
    M, K = A.shape
    rows = B.shape[0]
    if backward:
        F, n = rows, 2 * rows
    elif rows % 2:
        raise ValueError(f"B must have the gate's rows and as many of the up projection, got {tuple(B.shape)}")
    else:
        F = n = rows // 2
    mn = torch.Size((M, n))
    dt = D.dtype
    if dt in _U8:
        if d_fmt not in (E4M3, E5M2):
            raise ValueError("an FP8 output needs d_fmt (E4M3 or E5M2)")
        d_dtype = OUT_E4M3 if d_fmt == E4M3 else OUT_E5M2
    elif dt in _OUT:
        d_dtype = _OUT[dt]
    else:
        raise TypeError(f"D has dtype {dt}, expected bf16, float32 or FP8 codes")
    pt = _param_type(bias, dbias)
    kept = torch.Size((M, 2 * F))
    nkb = (K + 127) // 128 if M > 0 and F > 0 else 0
    on = A.get_device()
    ap, lda = _codes(A, A.shape, "A", on)
    bp, ldb = _codes(B, torch.Size((rows, K)), "B", on)
    dp, ldd = _mat(D, mn, dt, "D", on)
    tp, ldt = _codes(D_t, torch.Size((n, M)), "D_t", on) if D_t is not None else (0, M)
    ws, wp, wn = _workspace(workspace, lambda: fp8_gated_linear_workspace(M, F, K, a_scaling, b_scaling, backward), A,
                            stream, on)
    g = _pack_gemm(M, F, K, lda, ldb, ldd, ap, a_fmt, a_scaling, _scales(a_scale_inv, a_scaling, M, nkb, "a_scale_inv", on),
                   bp, b_fmt, b_scaling, _scales(b_scale_inv, b_scaling, rows, nkb, "b_scale_inv", on), dp, d_dtype,
                   _floats(d_amax, 1, "d_amax", on), 0, _floats(d_scale, 1, "d_scale", on), tp, ldt,
                   1 if amax_accumulate else 0)
    e = _pack_gated(1 if backward else 0, act, _DT[pt], _vec(bias, 2 * F, pt, "bias", on), *_mat(aux, kept, _BFLOAT, "aux", on),
                    *_codes(ck, kept, "ck", on), *_bytes(ck_exp, torch.Size((M, 2 * ((F + 31) // 32))), "ck_exp", on),
                    _vec(dbias, 2 * F, pt, "dbias", on), wp, wn)
    status = _L.fp8_gated_linear(g, e, _stream_on(on, stream))
    if status:
        _check("fp8_gated_linear", status)


def _bytes(t, shape, name, dev):
    """_mat of a checkpoint's powers of two (uint8 or float8_e8m0fnu)."""
    if t is not None and t.dtype not in _POWERS:
        raise TypeError(f"{name} has dtype {t.dtype}, expected uint8 or float8_e8m0fnu")
    return _mat(t, shape, None if t is None else t.dtype, name, dev)


def _checkpoint(x, ck, ck_exp, name):
    rows, cols = shape = _two_dim(x, name)
    if ck is None or ck_exp is None:
        raise ValueError("ck and ck_exp are required")
    nb, on = (cols + 31) // 32, x.get_device()
    if (ck.shape == shape and ck_exp.shape == (rows, nb) and ck.dtype in _U8 and ck_exp.dtype in _POWERS
            and 0 <= on == ck.get_device() == ck_exp.get_device() and x.is_contiguous() and ck.is_contiguous()
            and ck_exp.is_contiguous()):
        # (what most calls are; a small matrix's call is the host's time)
        return on, rows, cols, x.data_ptr(), cols, ck.data_ptr(), cols, ck_exp.data_ptr(), nb
    return (on, rows, cols, *_mat(x, shape, x.dtype, name, on), *_codes(ck, shape, "ck", on),
            *_bytes(ck_exp, torch.Size((rows, nb)), "ck_exp", on))


def fp8_checkpoint_save(x, ck, ck_exp, stream=None):
    """x [rows][cols], bf16 or float32, kept for the backward pass in 8 bits: ck
    [rows][cols] E4M3 codes (uint8 or float8) and ck_exp [rows][ceil(cols / 32)] one
    power of two for each 32 columns (uint8, or float8_e8m0fnu).  Rows may be strided."""
    on, rows, cols, xp, ldx, cp, ldc, ep, lde = _checkpoint(x, ck, ck_exp, "x")
    status = _L.fp8_checkpoint_save(xp, _DT[x.dtype], rows, cols, ldx, cp, ldc, ep, lde, _stream_on(on, stream))
    if status:
        _check("fp8_checkpoint_save", status)


def fp8_checkpoint_load(ck, ck_exp, y, stream=None):
    """y [rows][cols], bf16 or float32: the values of a checkpoint."""
    on, rows, cols, yp, ldy, cp, ldc, ep, lde = _checkpoint(y, ck, ck_exp, "y")
    status = _L.fp8_checkpoint_load(cp, ldc, ep, lde, rows, cols, yp, _DT[y.dtype], ldy, _stream_on(on, stream))
    if status:
        _check("fp8_checkpoint_load", status)


def fp8_rope_freqs(freqs, base=10000.0, scaling=ROPE_PLAIN, factor=1.0, trained=8192.0, low=1.0, high=32.0,
                   stream=None):
    """Rotation frequencies of freqs.numel() pairs (a float64 GPU tensor, filled
    here): base^(-i / pairs), scaled for contexts beyond the trained length by
    `scaling` (ROPE_PLAIN, ROPE_LINEAR, ROPE_BASE, ROPE_PARTS)."""
    _check("fp8_rope_freqs",
           _L.fp8_rope_freqs(_ptr(freqs, (torch.float64,), "freqs"), freqs.numel(), base, scaling, factor, trained,
                             low, high, _stream(stream)))


def _heads(t, shape, dtype, name, written=False):
    """(pointer, token stride, head stride) of [tokens][heads][dim] heads; heads
    that are written may not share memory."""
    if t.dtype != dtype or t.shape != shape or not t.is_cuda:
        _refuse(t, shape, dtype, name)
    ts, hs, one = t.stride()
    if one != 1 and shape[2] > 1:
        raise ValueError(f"{name} must have unit stride inside a head, got strides {t.stride()}")
    if written and ((ts == 0 and shape[0] > 1) or (hs == 0 and shape[1] > 1)):
        raise ValueError(f"{name} is written and must not be a broadcast view, got strides {t.stride()}")
    return t.data_ptr(), ts, hs


def fp8_rope(q, freqs, positions=None, k=None, q_out=None, k_out=None, layout=ROPE_HALF, inverse=False,
             scale=1.0, offset=0, stream=None):
    """Turns pair i of every head of q (and k) [tokens][heads][dim] by
    (position + offset) * freqs[i] and scales it; elements past the 2 *
    freqs.numel() turned ones are copied.  q and k may be strided views of one
    QKV tensor; without q_out / k_out they are turned in place.  positions:
    [tokens] int32 or int64 (None: 0, 1, ...).  inverse=True turns back: the
    gradient."""
    shape, dt = q.shape, q.dtype
    if dt not in _DT:
        raise TypeError(f"q must be bf16 or float32, got {dt}")
    if len(shape) != 3:
        raise ValueError(f"q must be [tokens][heads][dim], got {tuple(shape)}")
    tokens, qh, dim = shape
    qv = _heads(q, shape, dt, "q", q_out is None)
    qo = qv if q_out is None else _heads(q_out, shape, dt, "q_out", True)
    kh, kv, ko = 0, (0, 0, 0), (0, 0, 0)
    if k is not None:
        kshape = k.shape
        if len(kshape) != 3 or kshape[0] != tokens or kshape[2] != dim:
            raise ValueError(f"k must be [{tokens}][heads][{dim}], got {tuple(kshape)}")
        kh = kshape[1]
        kv = _heads(k, kshape, dt, "k", k_out is None)
        ko = kv if k_out is None else _heads(k_out, kshape, dt, "k_out", True)
    pp, wide = 0, 0
    if positions is not None:
        wide = 1 if positions.dtype == torch.int64 else 0
        pp = _vec(positions, tokens, torch.int64 if wide else torch.int32, "positions")
    pairs = freqs.numel()
    a = _pack_rope(tokens, qh, kh, dim, pairs, _DT[dt], layout, 1 if inverse else 0, scale,
                   _vec(freqs, pairs, torch.float64, "freqs"), pp, wide, offset, *qv, *kv, *qo, *ko)
    status = _L.fp8_rope(a, _stream(stream))
    if status:
        _check("fp8_rope", status)
