"""The low-precision operands' definitions in 64 bits (numpy): include/quant.h's formats bit
for bit, and the norm and the product with bounds on how far a 32-bit evaluation may be
from them (oracle/ffn.py says how such bounds are made).  No code is shared with the CUDA path.
"""
from __future__ import annotations

import collections

import numpy as np

from . import ffn

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
BLOCK = {"e4m3": 0, "mxe4m3": 32, "mxfp4": 32, "nvfp4": 16}
LARGEST = {"mxe4m3": 448.0, "mxfp4": 6.0, "nvfp4": 2688.0}


def _e4m3_table():
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v[b] = np.nan if b & 127 == 127 else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        if b & 128:
            v[b] = -v[b]
    return v


E4M3 = _e4m3_table()

# codes: uint8, a value a place; scales: uint8 (rows, scale columns) or None; row_scale: (rows) or None
Operand = collections.namedtuple("Operand", ["codes", "scales", "row_scale", "format", "cols"])


def width(cols):
    return max(32, -(-cols // 32) * 32)


def _nearest(t, table):
    """Codes of the nearest of table's values, ties to the even code; limited to the largest.
    `table`: ascending, from 0."""
    a = np.abs(t)
    i = np.clip(np.searchsorted(table, a, side="right") - 1, 0, len(table) - 2)
    low, high = table[i], table[i + 1]
    up = (a - low > high - a) | ((a - low == high - a) & (i % 2 == 1))
    return np.where(a >= table[-1], len(table) - 1, i + up).astype(np.uint8)


def e4m3(t):
    return _nearest(t, E4M3[:127]) | (np.signbit(t).astype(np.uint8) << 7)


def e2m1(t):
    return _nearest(t, E2M1[:8]) | (np.signbit(t).astype(np.uint8) << 3)


def covering(amax, largest):
    """The smallest whole e with amax <= largest * 2^e (amax > 0)."""
    m, e = np.frexp(amax)
    tm, te = np.frexp(largest)
    return e - te + (m > tm)


def quantise(x, fmt):
    """x (rows, cols) float64, of exact fp32 (or fp16, bf16) values: the Operand."""
    rows, cols = x.shape
    v = np.zeros((rows, width(cols)))
    v[:, :cols] = x
    fine = np.isfinite(v).all(1)
    if fmt == "e4m3":
        with np.errstate(invalid="ignore", over="ignore"):
            s = np.maximum(np.abs(v).max(1).astype(np.float32) / np.float32(448), np.float32(2.0 ** -126))
            t = v.astype(np.float32) * (np.float32(1) / s)[:, None]
        t[~fine] = 0
        s[~fine] = np.nan
        return Operand(e4m3(t.astype(np.float64)), None, s.astype(np.float64), fmt, cols)
    b = v.reshape(rows, v.shape[1] // BLOCK[fmt], BLOCK[fmt])
    if fmt == "nvfp4":
        b = np.where(fine[:, None, None], b, 0.0)
        top = np.abs(b).max((1, 2))
        row = np.ldexp(1.0, np.where(top > 0, np.maximum(covering(np.where(top > 0, top, 1.0), 2688.0), -100), 0))
        scales = e4m3(np.abs(b).max(2) / (6 * row[:, None]))
        unit = (E4M3[scales] * row[:, None])[:, :, None]
        codes = np.where(unit > 0, e2m1(b / np.where(unit > 0, unit, 1.0)), 0).astype(np.uint8)
        row[~fine], scales[~fine], codes[~fine] = np.nan, 127, 0
        return Operand(codes.reshape(v.shape), scales, row, fmt, cols)
    whole = np.isfinite(b).all(2)
    b = np.where(whole[:, :, None], b, 0.0)
    most = np.abs(b).max(2)
    e = np.where(most > 0, np.maximum(covering(np.where(most > 0, most, 1.0), LARGEST[fmt]), -127), -127)
    codes = (e4m3 if fmt == "mxe4m3" else e2m1)(b / np.ldexp(1.0, e)[:, :, None])
    codes[~whole] = 0
    return Operand(codes.reshape(v.shape), np.where(whole, e + 127, 255).astype(np.uint8), None, fmt, cols)


def tile(scales, rows):
    """The bytes of a scale array in the tiled order (include/quant.h), from the sentence alone."""
    cols = scales.shape[1]
    cb = -(-cols // 4)
    out = np.zeros(-(-rows // 128) * cb * 512, np.uint8)
    r, c = np.meshgrid(np.arange(rows), np.arange(cols), indexing="ij")
    out[((r // 128) * cb + c // 4) * 512 + (r % 32) * 16 + ((r // 32) % 4) * 4 + c % 4] = scales
    return out


def packed(codes):
    """Two 4-bit codes a byte, the first one low."""
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def unit(o):
    """What each code of a row is multiplied by."""
    rows, n = o.codes.shape
    u = np.ones((rows, n))
    if o.scales is not None:
        s = E4M3[o.scales] if o.format == "nvfp4" else np.where(o.scales == 255, np.nan, np.ldexp(1.0, o.scales.astype(int) - 127))
        u = u * np.repeat(s, BLOCK[o.format], 1)
    return u if o.row_scale is None else u * o.row_scale[:, None]


def values(o):
    """What an operand stands for, with its padding."""
    return (E2M1 if o.format in ("mxfp4", "nvfp4") else E4M3)[o.codes] * unit(o)


def product(a, b, dtype, bias=None, act="none", residual=None):
    """(c, bound) for operands a and b: exact products of 4-bit values, their sum in fp32 on the
    Tensor Core, an epilogue of a handful of fp32 operations, one rounding."""
    v, e = ffn.product(values(a), values(b))
    e = e + 3 * ffn.E * np.abs(v)
    if bias is not None:
        v = v + bias
        e = e + ffn.E * np.abs(v)
    if act != "none":
        g = v
        v, _ = ffn.activation(act, g)
        e = ffn.MAX_SLOPE * e + 2.0 ** -20 * (np.abs(v) if act == "relu" else 1 + np.abs(g)) * (act != "relu")
    if residual is not None:
        v = v + residual
    e = e + ffn.E * np.abs(v)
    return v, e + ffn.rounding(np.abs(v) + e, dtype)


def norm(y, residual, weight, dtype, eps, residual_scale=1.0, branch_scale=1.0):
    """((s, bound), (n, bound)): the stream, and the normalised values before they are quantised."""
    s = branch_scale * y + (0 if residual is None else residual_scale * residual)
    es = 2 * ffn.E * (np.abs(branch_scale * y) + (0 if residual is None else np.abs(residual_scale * residual)))
    u = ffn.Unit(s, es, "rms", eps)
    return (s, es + ffn.rounding(np.abs(s) + es, dtype)), u.affine(weight, None)


def half_step(codes, table):
    """Half the distance from each code's value to its farther neighbour."""
    mag = table[: (127 if len(table) == 256 else 8)]
    i = codes & (127 if len(table) == 256 else 7)
    up = np.where(i + 1 < len(mag), mag[np.minimum(i + 1, len(mag) - 1)] - mag[i], 0)
    down = np.where(i > 0, mag[i] - mag[np.maximum(i.astype(int) - 1, 0)], 0)
    return np.maximum(up, down) / 2
