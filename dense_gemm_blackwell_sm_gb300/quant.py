"""Binding of include/quant.h: low-precision operands and the 4-bit product (argument
marshalling and output allocation only).

    wq = quantise(w, "nvfp4")                            # a weight, once
    y = linear(x, wq, bias=b, act="silu")                # quantise(x), then the product
    s, nq = norm_quantise(y, s, weight, format="nvfp4")  # residual's addition, RMS norm, quantised
    y = product(nq, wq)
    dx, dw = linear_backward(dy, x, w, format="nvfp4")   # both products of the backward pass

Formats: "e4m3" (a float32 scale per row), "mxe4m3" (E4M3, a power of two per 32 elements),
"mxfp4" (E2M1, a power of two per 32) and "nvfp4" (E2M1, an E4M3 scale per 16 and a power of
two per row); include/quant.h defines them.  The products of the 8-bit ones are gemm.Plan's:
run_epilogue with scale_a and scale_b, and run_mx.  Rows are kept with their padding, so such a
plan is made for K = quant.width(columns).

Tensors are CUDA tensors whose rows are dense (last stride 1; the row pitch is free).  Work is
enqueued on ``stream`` (default: the current stream) of the tensors' device.  As in ``gemm``
and ``ffn``, every computation happens in libdgbgemm.so's kernels and there is no fallback.
``load`` and the structures give the same C functions to callers with addresses of their own.
"""
from __future__ import annotations

import collections
import ctypes

import torch

from . import ffn, gemm
from .ffn import ACTIVATIONS, _code, _share
from .gemm import GemmError

# quant_format_t
E4M3, MXE4M3, MXFP4, NVFP4 = 0, 1, 2, 3
FORMATS = {"e4m3": E4M3, "mxe4m3": MXE4M3, "mxfp4": MXFP4, "nvfp4": NVFP4}
_OUT = {torch.bfloat16: ffn.BF16, torch.float32: ffn.F32}

STATIC_B = 1
DEBUG_SKIP_ONE_LOAD = 1

_p, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class RowsArgs(ctypes.Structure):
    _fields_ = [("rows", _i64), ("cols", _i64), ("dtype", _i32), ("format", _i32), ("transpose", _i32),
                ("reserved", _i32), ("x", _p), ("data", _p), ("scales", _p), ("row_scale", _p), ("workspace", _p),
                ("ld_x", _i64), ("ld_data", _i64)]


class NormArgs(ctypes.Structure):
    _fields_ = [("M", _i64), ("D", _i64), ("dtype", _i32), ("param_dtype", _i32), ("format", _i32),
                ("reserved", _i32), ("eps", _f32), ("residual_scale", _f32), ("branch_scale", _f32),
                ("reserved_f", _f32), ("y", _p), ("residual", _p), ("weight", _p), ("s", _p), ("data", _p),
                ("scales", _p), ("row_scale", _p), ("ld_y", _i64), ("ld_residual", _i64), ("ld_s", _i64),
                ("ld_data", _i64)]


class ProductArgs(ctypes.Structure):
    _fields_ = [("M", _i64), ("N", _i64), ("K", _i64), ("format", _i32), ("out_dtype", _i32), ("activation", _i32),
                ("flags", _i32), ("a", _p), ("b", _p), ("scales_a", _p), ("scales_b", _p), ("row_scale_a", _p),
                ("row_scale_b", _p), ("bias", _p), ("residual", _p), ("c", _p), ("ld_a", _i64), ("ld_b", _i64),
                ("ld_residual", _i64), ("ld_c", _i64), ("timeout_ns", _i64), ("debug_flags", _i32),
                ("reserved", _i32 * 3)]


class LinearArgs(ctypes.Structure):
    _fields_ = [("M", _i64), ("N", _i64), ("K", _i64), ("dtype", _i32), ("format", _i32), ("out_dtype", _i32),
                ("activation", _i32), ("flags", _i32), ("debug_flags", _i32), ("x", _p), ("b", _p), ("scales_b", _p),
                ("row_scale_b", _p), ("bias", _p), ("residual", _p), ("c", _p), ("workspace", _p), ("ld_x", _i64),
                ("ld_b", _i64), ("ld_residual", _i64), ("ld_c", _i64), ("timeout_ns", _i64)]


class Quantised(collections.namedtuple("Quantised", ["data", "scales", "row_scale", "format", "cols"])):
    """A quantised operand: ``data`` (rows, row bytes), float8_e4m3fn or two 4-bit codes per
    byte (uint8); ``scales``, the tiled block scales' bytes, None for "e4m3"; ``row_scale``
    (rows) float32, None for the MX formats; ``format``, its name; ``cols``, the values of a
    row without their padding."""
    __slots__ = ()


_new = tuple.__new__  # (a call's five values are a Quantised's)

_lib = None


def load():
    """The library with this header's functions declared (raises if it is not built)."""
    global _lib
    if _lib is None:
        lib = gemm.load()
        for name, args in (("quant_rows", RowsArgs), ("quant_norm", NormArgs), ("quant_product", ProductArgs),
                           ("quant_linear", LinearArgs)):
            f = getattr(lib, name)
            f.argtypes, f.restype = [ctypes.POINTER(args), _p], ctypes.c_int  # (a structure is passed by reference)
        lib.quant_rows_many.argtypes, lib.quant_rows_many.restype = [ctypes.POINTER(RowsArgs), _i32, _p], ctypes.c_int
        lib.quant_rows_workspace.argtypes, lib.quant_rows_workspace.restype = [ctypes.POINTER(RowsArgs)], _i64
        lib.quant_linear_workspace.argtypes, lib.quant_linear_workspace.restype = [ctypes.POINTER(LinearArgs)], _i64
        lib.quant_width.argtypes, lib.quant_width.restype = [_i64], _i64
        lib.quant_row_bytes.argtypes, lib.quant_row_bytes.restype = [_i64, _i32], _i64
        lib.quant_scale_bytes.argtypes, lib.quant_scale_bytes.restype = [_i64, _i64, _i32], _i64
        lib.quant_check.argtypes, lib.quant_check.restype = [_p], ctypes.c_int
        _lib = lib
    return _lib


_calls = None


def load_calls():
    """The extension (raises if it is not built)."""
    global _calls
    if _calls is None:
        try:
            from . import _quant_calls
        except ImportError as e:
            raise RuntimeError("_quant_calls.so is not built (%s); run __graft_entry__.build() first" % e) from e
        _quant_calls.bind(GemmError, _share, FORMATS, tuple(FORMATS))
        _calls = _quant_calls
    return _calls


def _out_code(dtype):
    code = _OUT.get(dtype)
    if code is None:
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float32, not %s" % (dtype,))
    return code


def _values(q, name):
    """q itself: its five values are five arguments of a call."""
    if not isinstance(q, Quantised):
        raise TypeError("%s must be a Quantised, not %s" % (name, type(q).__name__))
    return q


def quantise(x, format, transpose=False, stream=None):
    """x (rows, cols), float16, bfloat16 or float32, quantised by rows, or with
    ``transpose`` by columns (the operand of x.T): a Quantised."""
    return _new(Quantised, (_calls or load_calls()).quantise(x, format, transpose, stream))


def norm_quantise(y, residual=None, weight=None, *, format, eps=1e-6, residual_scale=1.0, branch_scale=1.0,
                  need_s=True, s=None, stream=None):
    """The residual's addition and the RMS norm before the next layer, quantised by rows, in
    one kernel:

        s = residual_scale * residual + branch_scale * y
        n = s / sqrt(mean(s^2) + eps) * weight

    returns (s, Quantised of n), s None with need_s False.  s may be given, and be y or the
    residual (in place).  weight is (D), of y's type or float32.  Its gradient is that of
    ffn.block_norm with pre_weight=weight."""
    s, q = (_calls or load_calls()).norm_quantise(y, residual, weight, format, eps, residual_scale, branch_scale,
                                                  need_s, s, stream)
    return s, _new(Quantised, q)


def product(a, b, *, out_dtype=torch.bfloat16, bias=None, act="none", residual=None, out=None, static_b=False,
            stream=None, timeout_ns=0, debug_flags=0):
    """act(a @ b.T + bias) + residual for 4-bit operands a (M rows) and b (N rows) of one
    format and as many columns: (M, N), bfloat16 or float32.  bias is (N) float32, residual
    (M, N) of the output's type; it may be ``out``.  With ``static_b`` the kernel may read b
    while those before it on the stream still run: for weights, which these do not write."""
    return (_calls or load_calls()).product(*_values(a, "a"), *_values(b, "b"), _out_code(out_dtype), bias,
                                            _code(ACTIVATIONS, act, "act"), residual, out, static_b, stream,
                                            timeout_ns, debug_flags)


def linear(x, w, *, out_dtype=torch.bfloat16, bias=None, act="none", residual=None, out=None, static_b=False,
           stream=None, timeout_ns=0, debug_flags=0):
    """product(quantise(x, w.format), w, ...) for x (M, K) and a 4-bit weight w (N rows); up to 16
    tokens go in one kernel where that is as fast or faster with the launch it saves counted in.
    ``out`` must not share memory with x."""
    return (_calls or load_calls()).linear(x, *_values(w, "w"), _out_code(out_dtype), bias,
                                           _code(ACTIVATIONS, act, "act"), residual, out, static_b, stream,
                                           timeout_ns, debug_flags)


def linear_backward(dy, x, w, *, format, need_dx=True, need_dw=True, out_dtype=torch.bfloat16, stream=None,
                    timeout_ns=0):
    """(dx, dw) of y = x @ w.T for dy (M, N), x (M, K) and w (N, K), both products with 4-bit
    operands quantised along the sum: dx = Q(dy) Q(w^T)^T and dw = Q(dy^T) Q(x^T)^T.  The
    roundings are passed by: these are the gradients of the product of the unrounded values,
    made of rounded ones.  Either is None when not needed, and then its operand may be.

    It is the product's gradient alone: dy is what reaches x @ w.T.  Of ``linear``'s other parts the
    bias's gradient is dy's sum over the rows and the residual's is dy itself; with an activation
    dy has to have been multiplied by its derivative, for which a training step keeps what the
    activation is applied to (linear without ``act``, then the activation)."""
    return (_calls or load_calls()).linear_backward(dy, x, w, format, need_dx, need_dw, _out_code(out_dtype), stream,
                                                    timeout_ns)


def width(cols):
    """Elements of a quantised row of ``cols`` values (quant_width)."""
    return load().quant_width(int(cols))


def scale_bytes(rows, cols, format):
    """Bytes of the tiled block scales of ``rows`` rows of ``cols`` values (quant_scale_bytes)."""
    return load().quant_scale_bytes(int(rows), int(cols), _code(FORMATS, format, "format"))


def check(stream=None):
    """Synchronises the stream and returns gemm.OK, or the status of a device-side
    wait that ran out on the current device (quant_check)."""
    return load().quant_check(gemm._stream_ptr(stream))
