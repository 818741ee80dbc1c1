"""Binding of include/ffn.h: the feed-forward block's operators (argument
marshalling and output allocation only).

    h = gated(x, w, act="silu")                     # act(x Wg^T) * (x Wu^T), w = [Wg; Wu]
    h, gu = gated(x, w, act="silu", save=True)      # with the pre-activations, for training
    dx, dw = gated_backward(dh, x, w, gu=gu, act="silu")
    s, n = block_norm(y, residual, gate=g, pre_weight=w1, post_norm=True, post_weight=w2)
    grads = block_norm_backward(ds, dn, y, s, gate=g, ...)

Tensors are CUDA tensors whose rows are dense (last stride 1; the row pitch is
free).  Work is enqueued on ``stream`` (default: the current stream) of the
tensors' device.  As in ``gemm``, every computation happens in libdgbgemm.so's
kernels and there is no fallback.

The calls go through the extension _ffn_calls (csrc/ffn_python.cpp), since small
ones take longer in Python than on the device.  ``load`` and the structures give
the same C functions to callers with addresses of their own.
"""
from __future__ import annotations

import collections
import ctypes

import torch

from . import gemm
from .gemm import ACT_GELU_ERF, ACT_GELU_TANH, ACT_NONE, ACT_RELU, ACT_SILU, GemmError  # noqa: F401

# ffn_dtype_t
F16, BF16, F32 = 0, 1, 2

ACTIVATIONS = {"none": ACT_NONE, "relu": ACT_RELU, "silu": ACT_SILU, "gelu_tanh": ACT_GELU_TANH,
               "gelu_erf": ACT_GELU_ERF}

# ffn_norm_kind_t
NORM_RMS, NORM_LAYER = 0, 1
NORM_KINDS = {"rms": NORM_RMS, "layer": NORM_LAYER}

DEBUG_SKIP_ONE_LOAD = 1

_p, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class GatedArgs(ctypes.Structure):
    _fields_ = [("M", _i64), ("F", _i64), ("K", _i64), ("dtype", _i32), ("activation", _i32),
                ("x", _p), ("w", _p), ("h", _p), ("gu", _p),
                ("ld_x", _i64), ("ld_w", _i64), ("ld_h", _i64), ("ld_gu", _i64),
                ("timeout_ns", _i64), ("debug_flags", _i32), ("reserved", _i32 * 3)]


class GatedGradArgs(ctypes.Structure):
    _fields_ = [("M", _i64), ("F", _i64), ("K", _i64), ("dtype", _i32), ("activation", _i32),
                ("x", _p), ("w", _p), ("gu", _p), ("dh", _p), ("dgu", _p), ("dx", _p), ("dw", _p),
                ("workspace", _p), ("ld_x", _i64), ("ld_w", _i64), ("ld_gu", _i64), ("ld_dh", _i64), ("ld_dgu", _i64),
                ("ld_dx", _i64), ("ld_dw", _i64),
                ("timeout_ns", _i64), ("debug_flags", _i32), ("reserved", _i32 * 3)]


class NormArgs(ctypes.Structure):
    _fields_ = [("M", _i64), ("D", _i64), ("groups", _i64), ("dtype", _i32), ("param_dtype", _i32),
                ("kind", _i32), ("flags", _i32), ("eps", _f32), ("residual_scale", _f32), ("branch_scale", _f32),
                ("debug_flags", _i32),
                ("y", _p), ("residual", _p), ("gate", _p), ("post_weight", _p), ("post_bias", _p),
                ("pre_weight", _p), ("pre_bias", _p), ("s", _p), ("n", _p),
                ("ld_y", _i64), ("ld_residual", _i64), ("ld_gate", _i64), ("ld_s", _i64), ("ld_n", _i64)]


class NormGradArgs(ctypes.Structure):
    _fields_ = [("M", _i64), ("D", _i64), ("groups", _i64), ("dtype", _i32), ("param_dtype", _i32),
                ("kind", _i32), ("flags", _i32), ("eps", _f32), ("residual_scale", _f32), ("branch_scale", _f32),
                ("debug_flags", _i32),
                ("ds", _p), ("dn", _p), ("y", _p), ("s", _p), ("gate", _p), ("post_weight", _p),
                ("post_bias", _p), ("pre_weight", _p),
                ("dresidual", _p), ("dy", _p), ("dgate", _p), ("dpost_weight", _p), ("dpost_bias", _p),
                ("dpre_weight", _p), ("dpre_bias", _p), ("workspace", _p),
                ("ld_ds", _i64), ("ld_dn", _i64), ("ld_y", _i64), ("ld_s", _i64), ("ld_gate", _i64),
                ("ld_dresidual", _i64), ("ld_dy", _i64)]


# dresidual, dy: of the inputs' type; the parameters' gradients: fp32, None where the parameter is absent
NormGrads = collections.namedtuple("NormGrads", ["dresidual", "dy", "dgate", "dpost_weight", "dpost_bias",
                                                 "dpre_weight", "dpre_bias"])

_lib = None


def load():
    """The library with this header's functions declared (raises if it is not built)."""
    global _lib
    if _lib is None:
        lib = gemm.load()
        for name, args in (("ffn_gated", GatedArgs), ("ffn_gated_backward", GatedGradArgs), ("ffn_norm", NormArgs),
                           ("ffn_norm_backward", NormGradArgs)):
            f = getattr(lib, name)
            f.argtypes, f.restype = [ctypes.POINTER(args), _p], ctypes.c_int  # (a structure is passed by reference)
        for name, args in (("ffn_gated_backward_workspace", GatedGradArgs), ("ffn_norm_backward_workspace", NormGradArgs)):
            f = getattr(lib, name)
            f.argtypes, f.restype = [ctypes.POINTER(args)], _i64
        lib.ffn_check.argtypes, lib.ffn_check.restype = [_p], ctypes.c_int
        _lib = lib
    return _lib


_calls = None


def load_calls():
    """The extension (raises if it is not built)."""
    global _calls
    if _calls is None:
        try:
            from . import _ffn_calls
        except ImportError as e:
            raise RuntimeError("_ffn_calls.so is not built (%s); run __graft_entry__.build() first" % e) from e
        _ffn_calls.bind(GemmError, _share)
        _calls = _ffn_calls
    return _calls


def _code(table, value, what):
    code = table.get(value, value)
    if not isinstance(code, int):
        raise ValueError("%s must be one of %s" % (what, ", ".join(sorted(table))))
    return code


def _share(stream, index, tensors):
    """The handle of a given stream.  Memory allocated for a call belongs to the current
    stream: where the call goes to another one, that stream first waits for what may
    still use the memory, and the allocator is told of the use."""
    current = torch.cuda.current_stream(index)
    other = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=index)
    if other != current:
        other.wait_stream(current)
        for t in tensors:
            t.record_stream(other)
    return int(other.cuda_stream)


def gated(x, w, act="silu", save=False, out=None, gu=None, stream=None, timeout_ns=0, debug_flags=0):
    """h = act(x @ w[:F].T) * (x @ w[F:].T) for x (M, K) and w (2F, K), float16 or
    bfloat16, K a multiple of 8.

    ``act``: "none", "relu", "silu", "gelu_tanh", "gelu_erf" or a gemm.ACT_* code.
    With ``save`` the pre-activations (M, 2F) are kept for gated_backward and the
    answer is (h, gu).  ``out`` and ``gu`` may be given, as (M, F) and (M, 2F)."""
    h, gu = (_calls or load_calls()).gated(x, w, _code(ACTIVATIONS, act, "act"), save, out, gu, stream, timeout_ns,
                                            debug_flags)
    return (h, gu) if save else h


def gated_backward(dh, x, w, gu=None, act="silu", need_dx=True, need_dw=True, stream=None, timeout_ns=0,
                   debug_flags=0):
    """(dx, dw) of gated(x, w, act) for dh = dL/dh (M, F).  ``gu`` is what gated
    kept; without it the pre-activations are computed again from x and w.  dx
    (M, K) and dw (2F, K) have the inputs' type; either is None when not needed."""
    return (_calls or load_calls()).gated_backward(dh, x, w, gu, _code(ACTIVATIONS, act, "act"), need_dx, need_dw,
                                                    stream, timeout_ns, debug_flags)


def block_norm(y, residual=None, *, post_norm=False, post_weight=None, post_bias=None, gate=None, pre_norm=True,
               pre_weight=None, pre_bias=None, kind="rms", eps=1e-6, residual_scale=1.0, branch_scale=1.0,
               need_s=True, s=None, n=None, stream=None):
    """Merges a block's output y (M, D) into the residual stream and normalises the
    new stream for the next block, in one kernel:

        z = unit(y) * post_weight + post_bias  (post_norm)   or y
        s = residual_scale * residual + branch_scale * gate * z
        n = unit(s) * pre_weight + pre_bias    (pre_norm)

    and returns (s, n), None for a part not computed.  unit is the RMS norm
    (kind "rms") or the layer norm ("layer").  gate is (D), or (groups, D) with
    consecutive runs of M / groups rows sharing one.  s may be the residual and n
    may be y (in place).  Weights, biases and gate share one type, y's or float32."""
    return (_calls or load_calls()).block_norm(
        y, residual, post_norm, post_weight, post_bias, gate, pre_norm, pre_weight, pre_bias,
        _code(NORM_KINDS, kind, "kind"), eps, residual_scale, branch_scale, need_s, s, n, stream)


def block_norm_backward(ds, dn, y, s, *, post_norm=False, post_weight=None, post_bias=None, gate=None,
                        pre_norm=True, pre_weight=None, pre_bias=None, kind="rms", eps=1e-6, residual_scale=1.0,
                        branch_scale=1.0, need_dresidual=True, need_dy=True, need_dparams=True, stream=None):
    """NormGrads of block_norm for ds = dL/ds (None: zero) and dn = dL/dn, from its y
    and the s it returned.  A parameter's gradient (fp32) is computed where the
    parameter is given; dgate has the gate's shape."""
    return NormGrads._make((_calls or load_calls()).block_norm_backward(
        ds, dn, y, s, post_norm, post_weight, post_bias, gate, pre_norm, pre_weight, pre_bias,
        _code(NORM_KINDS, kind, "kind"), eps, residual_scale, branch_scale, need_dresidual, need_dy, need_dparams,
        stream))


def check(stream=None):
    """Synchronises the stream and returns gemm.OK, or the status of a device-side
    wait that ran out on the current device (ffn_check)."""
    return load().ffn_check(gemm._stream_ptr(stream))
