"""ctypes binding of include/ffn.h: the feed-forward block's operators (argument
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
"""
from __future__ import annotations

import collections
import ctypes

import torch

from . import gemm
from .gemm import ACT_GELU_ERF, ACT_GELU_TANH, ACT_NONE, ACT_RELU, ACT_SILU, GemmError  # noqa: F401

# ffn_dtype_t
F16, BF16, F32 = 0, 1, 2
_DTYPES = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}

ACTIVATIONS = {"none": ACT_NONE, "relu": ACT_RELU, "silu": ACT_SILU, "gelu_tanh": ACT_GELU_TANH,
               "gelu_erf": ACT_GELU_ERF}

# ffn_norm_kind_t
NORM_RMS, NORM_LAYER = 0, 1
NORM_KINDS = {"rms": NORM_RMS, "layer": NORM_LAYER}
_POST, _PRE = 1, 2

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
                ("ld_x", _i64), ("ld_w", _i64), ("ld_gu", _i64), ("ld_dh", _i64), ("ld_dgu", _i64),
                ("ld_dx", _i64), ("ld_dw", _i64),
                ("timeout_ns", _i64), ("debug_flags", _i32), ("reserved", _i32 * 3)]


class NormArgs(ctypes.Structure):
    _fields_ = [("M", _i64), ("D", _i64), ("groups", _i64), ("dtype", _i32), ("param_dtype", _i32),
                ("kind", _i32), ("flags", _i32), ("eps", _f32), ("residual_scale", _f32), ("branch_scale", _f32),
                ("reserved", _i32),
                ("y", _p), ("residual", _p), ("gate", _p), ("post_weight", _p), ("post_bias", _p),
                ("pre_weight", _p), ("pre_bias", _p), ("s", _p), ("n", _p),
                ("ld_y", _i64), ("ld_residual", _i64), ("ld_gate", _i64), ("ld_s", _i64), ("ld_n", _i64)]


class NormGradArgs(ctypes.Structure):
    _fields_ = [("M", _i64), ("D", _i64), ("groups", _i64), ("dtype", _i32), ("param_dtype", _i32),
                ("kind", _i32), ("flags", _i32), ("eps", _f32), ("residual_scale", _f32), ("branch_scale", _f32),
                ("reserved", _i32),
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
            f.argtypes, f.restype = [ctypes.POINTER(args), _p], ctypes.c_int
        lib.ffn_norm_backward_workspace.argtypes = [ctypes.POINTER(NormGradArgs)]
        lib.ffn_norm_backward_workspace.restype = _i64
        lib.ffn_check.argtypes, lib.ffn_check.restype = [_p], ctypes.c_int
        _lib = lib
    return _lib


def _matrix(name, t, rows, cols, like):
    """Checks a (rows x cols) tensor of `like`'s type and device with dense rows."""
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError("%s must be (%d, %d), not %s" % (name, rows, cols, tuple(t.shape)))
    if t.dtype != like.dtype or t.device != like.device:
        raise ValueError("%s must be %s on %s" % (name, like.dtype, like.device))
    if cols > 1 and t.stride(1) != 1 or rows > 1 and t.stride(0) < cols:
        raise ValueError("%s must have dense, non-overlapping rows" % name)
    return t


def _pitch(t):
    """The row pitch of a checked matrix (its length where there is no second row)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _code(table, value, what):
    code = table.get(value, value)
    if not isinstance(code, int):
        raise ValueError("%s must be one of %s" % (what, ", ".join(sorted(table))))
    return code


class _On:
    """The stream a call runs on.  Memory allocated for the call belongs to the
    current stream, so where the call goes to another one the allocator is told."""

    def __init__(self, device, stream):
        if device.type != "cuda":
            raise ValueError("tensors must be on a CUDA device")
        self.stream = stream
        self.other = stream is not None and stream != torch.cuda.current_stream(device)
        self.ptr = gemm._stream_ptr(stream if stream is not None else torch.cuda.current_stream(device))

    def empty(self, shape, dtype, device):
        t = torch.empty(shape, dtype=dtype, device=device)
        if self.other:
            self._order(t)
        return t

    def _order(self, t):
        # the memory may still be in use on the current stream
        current = torch.cuda.current_stream(t.device)
        stream = self.stream if hasattr(self.stream, "cuda_stream") else torch.cuda.ExternalStream(int(self.stream))
        stream.wait_stream(current)
        t.record_stream(stream)


def _call(name, args, device, on):
    fn = getattr(load(), name)
    if device.index == torch.cuda.current_device():
        status = fn(ctypes.byref(args), on.ptr)
    else:
        with torch.cuda.device(device):
            status = fn(ctypes.byref(args), on.ptr)
    if status != gemm.OK:
        raise GemmError(status, name)


def _gated_inputs(x, w):
    if x.dim() != 2 or w.dim() != 2 or w.shape[0] % 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x must be (M, K) and w (2F, K), not %s and %s" % (tuple(x.shape), tuple(w.shape)))
    M, K = x.shape
    F = w.shape[0] // 2
    _matrix("x", x, M, K, x)
    _matrix("w", w, 2 * F, K, x)
    if x.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("x must be float16 or bfloat16, not %s" % x.dtype)
    return M, F, K, _DTYPES[x.dtype]


def gated(x, w, act="silu", save=False, out=None, gu=None, stream=None, timeout_ns=0, debug_flags=0):
    """h = act(x @ w[:F].T) * (x @ w[F:].T) for x (M, K) and w (2F, K), float16 or
    bfloat16, K a multiple of 8.

    ``act``: "none", "relu", "silu", "gelu_tanh", "gelu_erf" or a gemm.ACT_* code.
    With ``save`` the pre-activations (M, 2F) are kept for gated_backward and the
    answer is (h, gu).  ``out`` and ``gu`` may be given, as (M, F) and (M, 2F)."""
    M, F, K, dtype = _gated_inputs(x, w)
    on = _On(x.device, stream)
    h = on.empty((M, F), x.dtype, x.device) if out is None else _matrix("out", out, M, F, x)
    if gu is not None:
        _matrix("gu", gu, M, 2 * F, x)
    elif save:
        gu = on.empty((M, 2 * F), x.dtype, x.device)
    args = GatedArgs(M, F, K, dtype, _code(ACTIVATIONS, act, "act"), x.data_ptr(), w.data_ptr(), h.data_ptr(),
                     gu.data_ptr() if gu is not None else None, _pitch(x), _pitch(w), _pitch(h),
                     _pitch(gu) if gu is not None else 0, timeout_ns, debug_flags)
    _call("ffn_gated", args, x.device, on)
    return (h, gu) if save else h


def gated_backward(dh, x, w, gu=None, act="silu", need_dx=True, need_dw=True, stream=None, timeout_ns=0,
                   debug_flags=0):
    """(dx, dw) of gated(x, w, act) for dh = dL/dh (M, F).  ``gu`` is what gated
    kept; without it the pre-activations are computed again from x and w.  dx
    (M, K) and dw (2F, K) have the inputs' type; either is None when not needed."""
    M, F, K, dtype = _gated_inputs(x, w)
    _matrix("dh", dh, M, F, x)
    if gu is not None:
        _matrix("gu", gu, M, 2 * F, x)
    on = _On(x.device, stream)
    ld_dgu = (2 * F + 7) // 8 * 8
    dgu = on.empty((M, ld_dgu), x.dtype, x.device)
    dx = on.empty((M, K), x.dtype, x.device) if need_dx else None
    dw = on.empty((2 * F, K), x.dtype, x.device) if need_dw else None
    args = GatedGradArgs(M, F, K, dtype, _code(ACTIVATIONS, act, "act"), x.data_ptr(), w.data_ptr(),
                         gu.data_ptr() if gu is not None else None, dh.data_ptr(), dgu.data_ptr(),
                         dx.data_ptr() if need_dx else None, dw.data_ptr() if need_dw else None,
                         _pitch(x), _pitch(w), _pitch(gu) if gu is not None else 0, _pitch(dh), ld_dgu, K, K,
                         timeout_ns, debug_flags)
    _call("ffn_gated_backward", args, x.device, on)
    return dx, dw


class _Norm:
    """The arguments block_norm and block_norm_backward share, checked."""

    def __init__(self, like, gate, vectors, kind, flags):
        if like.dim() != 2:
            raise ValueError("rows must be a 2-D tensor, not %s" % (tuple(like.shape),))
        self.M, self.D = like.shape
        self.dtype = _DTYPES.get(like.dtype)
        if self.dtype is None:
            raise ValueError("rows must be float16, bfloat16 or float32, not %s" % like.dtype)
        self.kind, self.flags = _code(NORM_KINDS, kind, "kind"), flags
        param = None
        for name, v in vectors:
            if v is not None:
                if v.dim() != 1 or v.shape[0] != self.D or (self.D > 1 and v.stride(0) != 1):
                    raise ValueError("%s must be %d dense values" % (name, self.D))
                param = self._param(name, v, param, like)
        self.gate, self.groups, self.ld_gate = None, 1, 0
        if gate is not None:
            g = gate.unsqueeze(0) if gate.dim() == 1 else gate
            param = self._param("gate", g, param, like)
            if g.dim() != 2 or g.shape[0] < 1 or self.M % g.shape[0]:
                raise ValueError("gate must be (D) or (groups, D) with the rows a multiple of the groups")
            _matrix("gate", g, g.shape[0], self.D, g)
            self.gate, self.groups, self.ld_gate = g.data_ptr(), g.shape[0], _pitch(g)
        self.param = _DTYPES[param] if param is not None else self.dtype

    @staticmethod
    def _param(name, v, param, like):
        if v.device != like.device or v.dtype not in (like.dtype, torch.float32) or param not in (None, v.dtype):
            raise ValueError("%s must be on %s, and weights, biases and gate all %s or all float32"
                             % (name, like.device, like.dtype))
        return v.dtype


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _ld(t):
    return _pitch(t) if t is not None else 0


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
    P = _Norm(y, gate, (("post_weight", post_weight), ("post_bias", post_bias), ("pre_weight", pre_weight),
                        ("pre_bias", pre_bias)), kind, (_POST if post_norm else 0) | (_PRE if pre_norm else 0))
    M, D = P.M, P.D
    _matrix("y", y, M, D, y)
    if residual is not None:
        _matrix("residual", residual, M, D, y)
    if not post_norm and (post_weight is not None or post_bias is not None):
        raise ValueError("post_weight and post_bias need post_norm")
    if not pre_norm and (pre_weight is not None or pre_bias is not None or n is not None):
        raise ValueError("pre_weight, pre_bias and n need pre_norm")
    on = _On(y.device, stream)
    if s is not None:
        _matrix("s", s, M, D, y)
    elif need_s:
        s = on.empty((M, D), y.dtype, y.device)
    if n is not None:
        _matrix("n", n, M, D, y)
    elif pre_norm:
        n = on.empty((M, D), y.dtype, y.device)
    args = NormArgs(M, D, P.groups, P.dtype, P.param, P.kind, P.flags, eps, residual_scale, branch_scale, 0,
                    y.data_ptr(), _ptr(residual), P.gate, _ptr(post_weight), _ptr(post_bias), _ptr(pre_weight),
                    _ptr(pre_bias), _ptr(s), _ptr(n), _pitch(y), _ld(residual), P.ld_gate, _ld(s), _ld(n))
    _call("ffn_norm", args, y.device, on)
    return s, n


def block_norm_backward(ds, dn, y, s, *, post_norm=False, post_weight=None, post_bias=None, gate=None,
                        pre_norm=True, pre_weight=None, pre_bias=None, kind="rms", eps=1e-6, residual_scale=1.0,
                        branch_scale=1.0, need_dresidual=True, need_dy=True, need_dparams=True, stream=None):
    """NormGrads of block_norm for ds = dL/ds (None: zero) and dn = dL/dn, from its y
    and the s it returned.  A parameter's gradient (fp32) is computed where the
    parameter is given; dgate has the gate's shape."""
    like = dn if dn is not None else ds
    if like is None:
        raise ValueError("ds or dn must be given")
    P = _Norm(like, gate, (("post_weight", post_weight), ("post_bias", post_bias), ("pre_weight", pre_weight),
                           ("pre_bias", pre_bias)), kind, (_POST if post_norm else 0) | (_PRE if pre_norm else 0))
    M, D = P.M, P.D
    if pre_norm and (dn is None or s is None) or not pre_norm and dn is not None:
        raise ValueError("dn and s are needed with pre_norm, and dn only then")
    if y is None and (post_norm or gate is not None and need_dparams):
        raise ValueError("y is needed with post_norm or a gate")
    if not post_norm and (post_weight is not None or post_bias is not None):
        raise ValueError("post_weight and post_bias need post_norm")
    if not pre_norm and (pre_weight is not None or pre_bias is not None):
        raise ValueError("pre_weight and pre_bias need pre_norm")
    for name, t in (("ds", ds), ("dn", dn), ("y", y), ("s", s)):
        if t is not None:
            _matrix(name, t, M, D, like)
    on = _On(like.device, stream)
    rows = lambda need: on.empty((M, D), like.dtype, like.device) if need else None  # noqa: E731
    sums = lambda p: (on.empty(p.shape, torch.float32, like.device)  # noqa: E731
                      if p is not None and need_dparams else None)
    g = NormGrads(rows(need_dresidual), rows(need_dy), sums(gate), sums(post_weight), sums(post_bias),
                  sums(pre_weight), sums(pre_bias))
    args = NormGradArgs(M, D, P.groups, P.dtype, P.param, P.kind, P.flags, eps, residual_scale, branch_scale, 0,
                        _ptr(ds), _ptr(dn), _ptr(y), _ptr(s), P.gate, _ptr(post_weight), _ptr(post_bias),
                        _ptr(pre_weight), *map(_ptr, g), None, _ld(ds), _ld(dn), _ld(y), _ld(s), P.ld_gate,
                        _ld(g.dresidual), _ld(g.dy))
    size = load().ffn_norm_backward_workspace(ctypes.byref(args))
    if size > 0:
        workspace = on.empty((size,), torch.uint8, like.device)
        args.workspace = workspace.data_ptr()
    _call("ffn_norm_backward", args, like.device, on)
    return g


def check(stream=None):
    """Synchronises the stream and returns gemm.OK, or the status of a device-side
    wait that ran out on the current device (ffn_check)."""
    return load().ffn_check(gemm._stream_ptr(stream))
