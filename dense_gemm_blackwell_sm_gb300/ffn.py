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

# the current stream's handle without a Stream object (torch's generated code uses it too)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)

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
        lib.ffn_norm_backward_workspace.argtypes = [ctypes.POINTER(NormGradArgs)]
        lib.ffn_norm_backward_workspace.restype = _i64
        lib.ffn_check.argtypes, lib.ffn_check.restype = [_p], ctypes.c_int
        _lib = lib
    return _lib


def _rows(name, t, shape, dtype, index):
    """Checks a CUDA tensor of dense rows on device `index` and returns their pitch."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        raise ValueError("%s must be %s of %s on cuda:%d, not %s of %s on %s"
                         % (name, tuple(shape), dtype, index, tuple(t.shape), t.dtype, t.device))
    if t.is_contiguous():
        return shape[1]
    rows, cols = shape
    pitch, step = t.stride()
    if cols > 1 and step != 1 or rows > 1 and pitch < cols:
        raise ValueError("%s must have dense, non-overlapping rows" % name)
    return pitch if rows > 1 else cols


def _device(t):
    index = t.get_device()
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    return index


def _code(table, value, what):
    code = table.get(value, value)
    if not isinstance(code, int):
        raise ValueError("%s must be one of %s" % (what, ", ".join(sorted(table))))
    return code


def _share(stream, index, tensors):
    """Memory allocated for a call belongs to the current stream: where the call goes
    to another one, that stream first waits for what may still use the memory, and the
    allocator is told of the use."""
    current = torch.cuda.current_stream(index)
    other = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=index)
    if other == current:
        return
    other.wait_stream(current)
    for t in tensors:
        if t is not None:
            t.record_stream(other)


def _call(fn, args, index, stream, made):
    if stream is None:
        ptr = _current_raw_stream(index)
    else:
        _share(stream, index, made)
        ptr = gemm._stream_ptr(stream)
    if index == _current_device():
        status = fn(args, ptr)
    else:
        with torch.cuda.device(index):
            status = fn(args, ptr)
    if status != gemm.OK:
        raise GemmError(status, fn.__name__)


def _gated_inputs(x, w):
    if x.dim() != 2 or w.dim() != 2 or w.shape[0] % 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x must be (M, K) and w (2F, K), not %s and %s" % (tuple(x.shape), tuple(w.shape)))
    dtype, index = x.dtype, _device(x)
    if dtype is not torch.float16 and dtype is not torch.bfloat16:
        raise ValueError("x must be float16 or bfloat16, not %s" % dtype)
    return (*x.shape, w.shape[0] // 2, dtype, index, _rows("x", x, x.shape, dtype, index),
            _rows("w", w, w.shape, dtype, index))


def gated(x, w, act="silu", save=False, out=None, gu=None, stream=None, timeout_ns=0, debug_flags=0):
    """h = act(x @ w[:F].T) * (x @ w[F:].T) for x (M, K) and w (2F, K), float16 or
    bfloat16, K a multiple of 8.

    ``act``: "none", "relu", "silu", "gelu_tanh", "gelu_erf" or a gemm.ACT_* code.
    With ``save`` the pre-activations (M, 2F) are kept for gated_backward and the
    answer is (h, gu).  ``out`` and ``gu`` may be given, as (M, F) and (M, 2F)."""
    M, K, F, dtype, index, ld_x, ld_w = _gated_inputs(x, w)
    device = x.device
    ld_h, ld_gu = F, 2 * F
    h = out
    if h is None:
        h = torch.empty((M, F), dtype=dtype, device=device)
    else:
        ld_h = _rows("out", h, (M, F), dtype, index)
    if gu is not None:
        ld_gu = _rows("gu", gu, (M, 2 * F), dtype, index)
    elif save:
        gu = torch.empty((M, 2 * F), dtype=dtype, device=device)
    args = GatedArgs(M, F, K, _DTYPES[dtype], _code(ACTIVATIONS, act, "act"), x.data_ptr(), w.data_ptr(),
                     h.data_ptr(), gu.data_ptr() if gu is not None else None, ld_x, ld_w, ld_h, ld_gu, timeout_ns,
                     debug_flags)
    _call((_lib or load()).ffn_gated, args, index, stream, (h, gu))
    return (h, gu) if save else h


def gated_backward(dh, x, w, gu=None, act="silu", need_dx=True, need_dw=True, stream=None, timeout_ns=0,
                   debug_flags=0):
    """(dx, dw) of gated(x, w, act) for dh = dL/dh (M, F).  ``gu`` is what gated
    kept; without it the pre-activations are computed again from x and w.  dx
    (M, K) and dw (2F, K) have the inputs' type; either is None when not needed."""
    M, K, F, dtype, index, ld_x, ld_w = _gated_inputs(x, w)
    device = x.device
    ld_dh = _rows("dh", dh, (M, F), dtype, index)
    ld_gu = _rows("gu", gu, (M, 2 * F), dtype, index) if gu is not None else 0
    ld_dgu = (2 * F + 7) // 8 * 8
    dgu = torch.empty((M, ld_dgu), dtype=dtype, device=device)
    dx = torch.empty((M, K), dtype=dtype, device=device) if need_dx else None
    dw = torch.empty((2 * F, K), dtype=dtype, device=device) if need_dw else None
    args = GatedGradArgs(M, F, K, _DTYPES[dtype], _code(ACTIVATIONS, act, "act"), x.data_ptr(), w.data_ptr(),
                         gu.data_ptr() if gu is not None else None, dh.data_ptr(), dgu.data_ptr(),
                         dx.data_ptr() if need_dx else None, dw.data_ptr() if need_dw else None,
                         ld_x, ld_w, ld_gu, ld_dh, ld_dgu, K, K, timeout_ns, debug_flags)
    _call((_lib or load()).ffn_gated_backward, args, index, stream, (dgu, dx, dw))
    return dx, dw


def _like(t, shape):
    """A dense tensor of t's type and shape."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(shape, dtype=t.dtype, device=t.device)


def _norm_parameters(like, gate, post_weight, post_bias, pre_weight, pre_bias, post_norm, pre_norm):
    """Checks what block_norm and its gradient share: (M, D, type, parameter type,
    the gate's pointer, groups and pitch, the vectors' pointers)."""
    if like.dim() != 2:
        raise ValueError("rows must be a 2-D tensor, not %s" % (tuple(like.shape),))
    M, D = like.shape
    dtype, index, param = like.dtype, _device(like), None
    if dtype not in _DTYPES:
        raise ValueError("rows must be float16, bfloat16 or float32, not %s" % dtype)
    if not post_norm and (post_weight is not None or post_bias is not None):
        raise ValueError("post_weight and post_bias need post_norm")
    if not pre_norm and (pre_weight is not None or pre_bias is not None):
        raise ValueError("pre_weight and pre_bias need pre_norm")
    gate_ptr, groups, ld_gate = None, 1, D
    if gate is not None:
        param = gate.dtype
        g = gate.unsqueeze(0) if gate.dim() == 1 else gate
        groups = g.shape[0]
        if g.dim() != 2 or groups < 1 or M % groups:
            raise ValueError("gate must be (D) or (groups, D) with the rows a multiple of the groups")
        ld_gate = _rows("gate", g, (groups, D), param, index)
        gate_ptr = g.data_ptr()
    ptrs = []
    for v in (post_weight, post_bias, pre_weight, pre_bias):
        if v is None:
            ptrs.append(None)
            continue
        if param is None:
            param = v.dtype
        if v.shape != (D,) or v.dtype is not param or v.get_device() != index or not v.is_contiguous():
            raise ValueError("weights and biases must be %d dense values of %s on cuda:%d" % (D, param, index))
        ptrs.append(v.data_ptr())
    if param is None:
        param = dtype
    elif param is not dtype and param is not torch.float32:
        raise ValueError("weights, biases and gate must be %s or float32, not %s" % (dtype, param))
    return M, D, dtype, index, _DTYPES[dtype], _DTYPES[param], gate_ptr, groups, ld_gate, ptrs


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
    M, D, dtype, index, code, param, gate_ptr, groups, ld_gate, p = _norm_parameters(
        y, gate, post_weight, post_bias, pre_weight, pre_bias, post_norm, pre_norm)
    shape = (M, D)
    ld_y = _rows("y", y, shape, dtype, index)
    res_ptr = s_ptr = n_ptr = None
    ld_res = ld_s = ld_n = D
    if residual is not None:
        ld_res = _rows("residual", residual, shape, dtype, index)
        res_ptr = residual.data_ptr()
    if s is not None:
        ld_s = _rows("s", s, shape, dtype, index)
    elif need_s:
        s = _like(y, shape)
    if n is not None:
        if not pre_norm:
            raise ValueError("n needs pre_norm")
        ld_n = _rows("n", n, shape, dtype, index)
    elif pre_norm:
        n = _like(y, shape)
    if s is not None:
        s_ptr = s.data_ptr()
    if n is not None:
        n_ptr = n.data_ptr()
    args = NormArgs(M, D, groups, code, param, _code(NORM_KINDS, kind, "kind"),
                    (_POST if post_norm else 0) | (_PRE if pre_norm else 0), eps, residual_scale, branch_scale, 0,
                    y.data_ptr(), res_ptr, gate_ptr, p[0], p[1], p[2], p[3], s_ptr, n_ptr, ld_y, ld_res, ld_gate,
                    ld_s, ld_n)
    _call((_lib or load()).ffn_norm, args, index, stream, (s, n))
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
    if pre_norm and (dn is None or s is None) or not pre_norm and dn is not None:
        raise ValueError("dn and s are needed with pre_norm, and dn only then")
    if y is None and (post_norm or gate is not None and need_dparams):
        raise ValueError("y is needed with post_norm or a gate")
    M, D, dtype, index, code, param, gate_ptr, groups, ld_gate, p = _norm_parameters(
        like, gate, post_weight, post_bias, pre_weight, pre_bias, post_norm, pre_norm)
    shape = (M, D)
    ins, lds = [], []
    for name, t in (("ds", ds), ("dn", dn), ("y", y), ("s", s)):
        lds.append(_rows(name, t, shape, dtype, index) if t is not None else D)
        ins.append(t.data_ptr() if t is not None else None)
    empty, device = torch.empty, like.device
    g = [_like(like, shape) if need_dresidual else None, _like(like, shape) if need_dy else None]
    for t in (gate, post_weight, post_bias, pre_weight, pre_bias):
        g.append(empty(t.shape, dtype=torch.float32, device=device) if t is not None and need_dparams else None)
    outs = [t.data_ptr() if t is not None else None for t in g]
    args = NormGradArgs(M, D, groups, code, param, _code(NORM_KINDS, kind, "kind"),
                        (_POST if post_norm else 0) | (_PRE if pre_norm else 0), eps, residual_scale, branch_scale, 0,
                        *ins, gate_ptr, p[0], p[1], p[2], *outs, None, *lds, ld_gate, D, D)
    workspace = None
    size = (_lib or load()).ffn_norm_backward_workspace(args)
    if size > 0:
        workspace = empty(size, dtype=torch.uint8, device=device)
        args.workspace = workspace.data_ptr()
    _call((_lib or load()).ffn_norm_backward, args, index, stream, (*g, workspace))
    return NormGrads(*g)


def check(stream=None):
    """Synchronises the stream and returns gemm.OK, or the status of a device-side
    wait that ran out on the current device (ffn_check)."""
    return load().ffn_check(gemm._stream_ptr(stream))
