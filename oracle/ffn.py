"""The feed-forward block's operators in 64 bits (numpy), with bounds on how far a
32-bit evaluation that rounds its outputs once may be from them.

The definitions are include/ffn.h's.  Every function returns (value, bound) pairs
or takes numpy float64 arrays of the exact inputs; no code is shared with the CUDA
path.  Bounds are derived here, from the number formats and the lengths of the
sums alone:

  E = 2^-24, the relative error of one fp32 operation;
  a product's sum over K terms on the Tensor Core: 16 terms are added per step of
    the accumulator, which may truncate, so K / 16 steps lose at most 2^-23 of the
    running absolute sum each; (K / 8 + 8) 2^-23 S covers that, the order of the
    16 and a CUDA-core sum in as many steps (S: the sum of absolute products);
  a row's sum over D elements: at most D / 128 + 16 additions follow one another
    in any of the kernels (threads add strided parts, then a tree);
  activations and their slopes: 2^-20 (1 + |g|) times their largest slope, the
    bound of the approximate exp2 and reciprocal with a factor to spare.
"""
from __future__ import annotations

import numpy as np
from scipy.special import erfc

E = 2.0 ** -24
FORMATS = {"bf16": (7, -126), "f16": (10, -14), "f32": (23, -126)}  # stored mantissa bits, smallest normal exponent
MAX_SLOPE, MAX_CURVE = 1.13, 1.2  # of every activation here but the step of ReLU's slope


def rounding(v, dtype):
    """Largest error of one rounding of values up to this size to dtype: half the
    spacing of the format there."""
    bits, smallest = FORMATS[dtype]
    with np.errstate(divide="ignore"):
        exponent = np.maximum(np.floor(np.log2(np.abs(v))), smallest)
    return 2.0 ** (exponent - bits - 1)


def activation(name, g):
    """act(g) and act'(g)."""
    if name == "none":
        return g.copy(), np.ones_like(g)
    if name == "relu":
        return np.maximum(g, 0.0), (g > 0).astype(np.float64)
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if name == "gelu_tanh":
        k = np.sqrt(2.0 / np.pi)
        t = np.tanh(k * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * g ** 2)
    p = 0.5 * erfc(-g / np.sqrt(2.0))
    return g * p, p + g * np.exp(-0.5 * g * g) / np.sqrt(2.0 * np.pi)


def product(a, b):
    """a @ b.T and the bound of its fp32 sum."""
    return a @ b.T, (a.shape[1] / 8 + 8) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)


def gated(x, w, act, dtype):
    """((h, bound), (gu, bound)) of the gated projections."""
    F = w.shape[0] // 2
    gu, e = product(x, w)
    g, u, eg, eu = gu[:, :F], gu[:, F:], e[:, :F], e[:, F:]
    a, _ = activation(act, g)
    ea = MAX_SLOPE * eg + 2.0 ** -20 * (1 + np.abs(g))
    h = a * u
    eh = ea * np.abs(u) + np.abs(a) * eu + ea * eu + 2 * E * np.abs(h)
    return (h, eh + rounding(np.abs(h) + eh, dtype)), (gu, e + rounding(np.abs(gu) + e, dtype))


def gated_backward(dh, x, w, gu, act, dtype):
    """((dx, bound), (dw, bound)); gu None: computed again from x and w."""
    F = w.shape[0] // 2
    if gu is None:
        gu, e = product(x, w)
    else:
        e = np.zeros_like(gu)
    g, u, eg, eu = gu[:, :F], gu[:, F:], e[:, :F], e[:, F:]
    a, d = activation(act, g)
    ea = MAX_SLOPE * eg + 2.0 ** -20 * (1 + np.abs(g))
    ed = MAX_CURVE * eg + 2.0 ** -19 * (1 + np.abs(g))
    if act == "relu":
        ed = np.where(np.abs(g) <= eg, 1.0, 0.0)  # a step: either side of it within the sum's error
    dgu = np.concatenate([dh * u * d, dh * a], 1)
    edgu = np.concatenate([np.abs(dh) * (np.abs(u) * ed + eu * np.abs(d) + eu * ed), np.abs(dh) * ea], 1)
    edgu += 3 * E * np.abs(dgu)
    edgu += rounding(np.abs(dgu) + edgu, dtype)
    out = []
    for left, e_left, right in ((dgu, edgu, w.T), (dgu.T, edgu.T, x.T)):
        v, ev = product(left, right)
        ev = ev * 1.01 + e_left @ np.abs(right).T
        out.append((v, ev + rounding(np.abs(v) + ev, dtype)))
    return tuple(out)


class Unit:
    """A row norm's values u = (v - mean) r, for v known to within `ev`."""

    def __init__(self, v, ev, kind, eps):
        D = v.shape[1]
        n = (D / 128 + 16) * E  # relative error of a row's sum of one sign
        m = lambda x: x.mean(1, keepdims=True)  # noqa: E731
        mean = m(v) if kind == "layer" else np.zeros((v.shape[0], 1))
        emean = (n + 2 * E) * m(np.abs(v)) + m(ev) if kind == "layer" else 0.0
        c = v - mean
        ec = emean + ev + E * np.abs(c)
        var = m(c * c)
        self.r = 1.0 / np.sqrt(var + eps)
        # r moves by half the relative change of var + eps: 2 c ec + ec^2 per element, plus the sum's error
        rel = 0.5 * (m(2 * np.abs(c) * ec + ec * ec) + (n + 4 * E) * var) * self.r ** 2 + 4 * E
        self.u = c * self.r
        self.er = self.r * rel * 1.01
        self.eu = ec * self.r + np.abs(c) * self.er + ec * self.er + E * np.abs(self.u)

    def affine(self, weight, bias):
        w = 1.0 if weight is None else weight
        v = self.u * w + (0.0 if bias is None else bias)
        return v, self.eu * np.abs(w) + 2 * E * (np.abs(self.u * w) + np.abs(v))

    def gradient(self, d, ed, weight, kind):
        """Gradient at v, with its bound, for the gradient d (known to within ed) of the affine result."""
        D = d.shape[1]
        n = (D / 128 + 16) * E
        m = lambda x: x.mean(1, keepdims=True)  # noqa: E731
        w = 1.0 if weight is None else weight
        a, ea = d * w, ed * np.abs(w) + E * np.abs(d * w)
        u, eu = self.u, self.eu
        mau = m(a * u)
        emau = m(np.abs(a) * eu + ea * np.abs(u) + ea * eu) + (n + 4 * E) * m(np.abs(a * u))
        ma = m(a) if kind == "layer" else 0.0
        ema = m(ea) + (n + 4 * E) * m(np.abs(a)) if kind == "layer" else 0.0
        q = a - u * mau - ma
        size = np.abs(a) + np.abs(u * mau) + np.abs(ma)
        eq = ea + eu * np.abs(mau) + np.abs(u) * emau + eu * emau + ema + 4 * E * size
        return self.r * q, self.r * eq + self.er * (np.abs(q) + eq) + 2 * E * np.abs(self.r * q)


def _per_row(gate, M):
    return np.ones((1, 1)) if gate is None else np.repeat(gate, M // gate.shape[0], 0)


def block_norm(y, residual, dtype, post, post_weight, post_bias, gate, pre, pre_weight, pre_bias, kind, eps,
               residual_scale=1.0, branch_scale=1.0):
    """((s, bound), (n, bound) or None)."""
    M = y.shape[0]
    z, ez = y, np.zeros_like(y)
    if post:
        z, ez = Unit(y, ez, kind, eps).affine(post_weight, post_bias)
    f = _per_row(gate, M) * branch_scale
    z, ez = f * z, np.abs(f) * ez + 2 * E * np.abs(f * z)
    res = np.zeros_like(y) if residual is None else residual_scale * residual
    s = res + z
    es = ez + 2 * E * (np.abs(res) + np.abs(z) + ez)
    first = (s, es + rounding(np.abs(s) + es, dtype))
    if not pre:
        return first, None
    n, en = Unit(s, es, kind, eps).affine(pre_weight, pre_bias)
    return first, (n, en + rounding(np.abs(n) + en, dtype))


def block_norm_backward(ds, dn, y, s, dtype, post, post_weight, post_bias, gate, pre, pre_weight, pre_bias, kind,
                        eps, residual_scale=1.0, branch_scale=1.0):
    """(value, bound) of dresidual, dy, dgate, dpost_weight, dpost_bias, dpre_weight,
    dpre_bias, None where the parameter is absent."""
    like = dn if dn is not None else ds
    M, D = like.shape
    zero = np.zeros_like(like)
    # a sum over M rows: rows of one thread follow one another, then the threads' and the CTAs' sums
    rows = (M + 64) * E

    def total(v, ev, groups=1):
        shape = (groups, M // groups, D)
        sums = v.reshape(shape).sum(1)
        bound = ev.reshape(shape).sum(1) * 1.01 + rows * np.abs(v).reshape(shape).sum(1)
        return (sums, bound + E * np.abs(sums)) if groups > 1 else (sums[0], (bound + E * np.abs(sums))[0])

    t, et = (zero if ds is None else ds), zero
    dpre_w = dpre_b = None
    if pre:
        unit = Unit(s, zero, kind, eps)
        v, ev = unit.gradient(dn, zero, pre_weight, kind)
        t, et = t + v, ev + 2 * E * (np.abs(t) + np.abs(v) + ev)
        if pre_weight is not None:
            dpre_w = total(dn * unit.u, np.abs(dn) * unit.eu + E * np.abs(dn * unit.u))
        if pre_bias is not None:
            dpre_b = total(dn, zero)
    f = _per_row(gate, M) * branch_scale
    dz, edz = f * t, np.abs(f) * et + 2 * E * np.abs(f) * (np.abs(t) + et)
    dy, edy = dz, edz
    z, ez = y, zero
    dpost_w = dpost_b = None
    if post:
        unit = Unit(y, zero, kind, eps)
        z, ez = unit.affine(post_weight, post_bias)
        dy, edy = unit.gradient(dz, edz, post_weight, kind)
        if post_weight is not None:
            dpost_w = total(dz * unit.u, np.abs(dz) * unit.eu + edz * (np.abs(unit.u) + unit.eu) +
                            E * np.abs(dz * unit.u))
        if post_bias is not None:
            dpost_b = total(dz, edz)
    dgate = None
    if gate is not None:
        b = abs(branch_scale)
        v, ev = total(branch_scale * t * z, b * (np.abs(t) * ez + et * (np.abs(z) + ez) + 3 * E * np.abs(t * z)),
                      gate.shape[0])
        dgate = (v.reshape(gate.shape), ev.reshape(gate.shape))
    dres, edres = residual_scale * t, abs(residual_scale) * et + 2 * E * np.abs(residual_scale * t)
    return ((dres, edres + rounding(np.abs(dres) + edres, dtype)), (dy, edy + rounding(np.abs(dy) + edy, dtype)),
            dgate, dpost_w, dpost_b, dpre_w, dpre_b)


def outside(got, ref):
    """(how many elements lie outside the bound, the worst error over its bound)."""
    value, bound = ref
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == value.shape, (got.shape, value.shape)
    with np.errstate(invalid="ignore", divide="ignore"):
        ratio = np.where(got == value, 0.0, np.abs(got - value) / bound)
    bad = ~(ratio <= 1.0)
    return int(bad.sum()), float(np.nanmax(ratio)) if ratio.size else 0.0
