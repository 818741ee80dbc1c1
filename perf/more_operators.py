"""Low-precision operands and what is done with them, as measured cases: quantisation to
8 and 4 bits (rows, or columns for the products of a backward pass), the residual's
addition with the RMS norm and an output in 8 bits with scales, the product of two
microscaled 4-bit operands, a linear layer that quantises its activations, and its
backward pass.

Formats: "e4m3" (a float32 scale per row), "mxe4m3" (E4M3 elements, a power of two per 32),
"mxfp4" (E2M1 elements, a power of two per 32), "nvfp4" (E2M1 elements, an E4M3 scale per
16 and a power of two per row).

``own`` False: elementary torch operations in 32 bits, rounded once at the end.
``own`` True: the calls a user makes of dense_gemm_blackwell_sm_gb300.quant.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
LARGEST = {"mxe4m3": (0.875, 9), "mxfp4": (0.75, 3), "nvfp4": (0.65625, 12)}  # as frexp gives 448, 6, 448 * 6


def listed():
    return [
        # a prompt's activations on their way into the block-scaled 8-bit product
        {"name": "quantise prompt 8192x4096 bf16", "op": "quantise", "rows": 8192, "cols": 4096, "dtype": "bf16",
         "format": "mxe4m3", "transpose": False},
        # a ragged half-precision batch with a width that fills no whole block, one scale per row
        {"name": "quantise ragged 777x1001 f16", "op": "quantise", "rows": 777, "cols": 1001, "dtype": "f16",
         "format": "e4m3", "transpose": False},
        # a weight's columns, the operand of the gradient with respect to the layer's input
        {"name": "quantise columns 14336x4096 bf16", "op": "quantise", "rows": 14336, "cols": 4096, "dtype": "bf16",
         "format": "mxe4m3", "transpose": True},
        # one decoded token between two blocks: pure latency
        {"name": "norm token 1x4096 bf16", "op": "norm", "M": 1, "D": 4096, "dtype": "bf16", "param": "bf16",
         "format": "e4m3"},
        # a prompt between two blocks
        {"name": "norm prompt 8192x4096 bf16", "op": "norm", "M": 8192, "D": 4096, "dtype": "bf16", "param": "f32",
         "format": "mxe4m3"},
        # a prompt through the largest projection shape, both operands quantised before: compute bound
        {"name": "product 8192x14336x4096 nvfp4", "op": "product", "M": 8192, "N": 14336, "K": 4096,
         "format": "nvfp4", "out": "bf16"},
        # a training batch too small to fill the card with large tiles
        {"name": "product 1024x1024x4096 mxfp4", "op": "product", "M": 1024, "N": 1024, "K": 4096,
         "format": "mxfp4", "out": "bf16"},
        # one decoded token through the largest projection shape: the weight stream and launches are all there is
        {"name": "linear token 1x14336x4096 nvfp4", "op": "linear", "M": 1, "N": 14336, "K": 4096, "dtype": "bf16",
         "format": "nvfp4", "act": "none", "fused": False, "out": "bf16"},
        # a decode batch of eight, with bias and activation
        {"name": "linear batch 8x4096x4096 mxfp4", "op": "linear", "M": 8, "N": 4096, "K": 4096, "dtype": "f16",
         "format": "mxfp4", "act": "silu", "fused": True, "out": "bf16"},
        # a short ragged batch of a small model: odd sizes, bias and activation, single precision out
        {"name": "linear ragged 300x1541x520 nvfp4", "op": "linear", "M": 300, "N": 1541, "K": 520, "dtype": "f32",
         "format": "nvfp4", "act": "relu", "fused": True, "out": "f32"},
        # a training batch's backward pass through the projection shape: compute bound, five arrays quantised
        {"name": "grad 4096x14336x4096 nvfp4", "op": "grad", "M": 4096, "N": 14336, "K": 4096, "dtype": "bf16",
         "format": "nvfp4"},
        # backward of a small odd-sized layer, half precision in
        {"name": "grad 515x1097x1032 mxfp4", "op": "grad", "M": 515, "N": 1097, "K": 1032, "dtype": "f16",
         "format": "mxfp4"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "norm", "product", "linear", "grad"])
    four = rng.choice(["mxfp4", "nvfp4"])
    if op == "quantise":
        rows = _log(rng, 1, 16384)
        return {"op": op, "rows": rows, "cols": _log(rng, 64, 14336 if rows <= 4096 else 4096),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "format": rng.choice(["e4m3", "mxe4m3"]),
                "transpose": rng.random() < 0.4}
    if op == "norm":
        M = _log(rng, 1, 8192)
        return {"op": op, "M": M, "D": _log(rng, 64, 8192 if M <= 4096 else 4096),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "param": "f32", "format": rng.choice(["e4m3", "mxe4m3"])}
    if op == "product":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 256, 14336), "K": 32 * _log(rng, 8, 128),
                "format": four, "out": "bf16"}
    if op == "linear":
        out = rng.choice(["bf16", "bf16", "f32"])
        return {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 256, 14336),
                "K": _log(rng, 256, 4096 if out == "bf16" else 1024), "dtype": rng.choice(["bf16", "f16", "f32"]),
                "format": four, "act": rng.choice(["none", "silu", "gelu_tanh", "relu"]),
                "fused": rng.random() < 0.5, "out": out}
    return {"op": op, "M": _log(rng, 64, 4096), "N": _log(rng, 256, 14336), "K": _log(rng, 256, 4096),
            "dtype": rng.choice(["bf16", "f16"]), "format": four}


def _up(n, m):
    return (n + m - 1) // m * m


def _held(rows, cols, fmt):
    """Bytes of a quantised operand: its elements and its scales."""
    n = rows * cols
    return {"e4m3": n + 4 * rows, "mxe4m3": n + n // 32, "mxfp4": n // 2 + n // 32,
            "nvfp4": n // 2 + n // 16 + 4 * rows}[fmt]


def work(case):
    c = case
    e = 4 if c.get("dtype") == "f32" else 2
    if c["op"] == "quantise":
        n = c["rows"] * c["cols"]
        rows, cols = (c["cols"], c["rows"]) if c["transpose"] else (c["rows"], c["cols"])
        return {"bytes": n * e + _held(rows, cols, c["format"]), "flops": 3 * n}
    if c["op"] == "norm":
        n = c["M"] * c["D"]
        return {"bytes": 3 * n * e + c["D"] * (4 if c["param"] == "f32" else 2) + _held(c["M"], c["D"], c["format"]),
                "flops": 9 * n}
    M, N, K = c["M"], c["N"], c["K"]
    if c["op"] == "grad":
        # dy, x and w read, dx and dw written
        return {"bytes": e * (M * N + M * K + N * K) + 2 * (M * K + N * K), "flops": 4 * M * N * K}
    a = _held(M, K, c["format"]) if c["op"] == "product" else M * K * e
    o = 4 if c["out"] == "f32" else 2
    fused = M * N * o + 4 * N if c.get("fused") else 0
    return {"bytes": a + _held(N, K, c["format"]) + M * N * o + fused, "flops": 2 * M * N * K}


# ------------------------------------------------- quantisation, elementary operations


def _pow2(e):
    """2^e for whole e of -127 to 127, from its bits (pow and ldexp may be off by one on a GPU)."""
    return torch.where(e >= -126, (e.int() + 127) << 23, 1 << 22).int().view(torch.float32)


def _exponent(amax, fmt):
    """The smallest e with amax <= largest * 2^e."""
    m, e = torch.frexp(amax)
    top, shift = LARGEST[fmt]
    return e - shift + (m > top).to(e.dtype)


def _e2m1(t):
    """The nearest of 0, 0.5, 1, 1.5, 2, 3, 4 and 6 (ties to the even code), with the sign."""
    a = t.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(t.dtype)
    return torch.copysign((torch.round(a / step) * step).clamp(max=6), t)


def _split(v, fmt):
    """v's rows (32 bits), padded with zeros to a multiple of 32, as (values, block scales,
    row scales): values in units of their scales; scales as values, None where there are none."""
    rows, cols = v.shape
    width = max(32, _up(cols, 32))
    v = torch.nn.functional.pad(v, (0, width - cols))
    if fmt == "e4m3":
        scale = (v.abs().amax(1) / 448).clamp(min=2.0 ** -126)
        return (v * (1 / scale)[:, None]).to(torch.float8_e4m3fn), None, scale
    if fmt == "nvfp4":
        amax = v.abs().amax(1)
        row = _pow2(torch.where(amax == 0, 0, _exponent(amax, fmt).clamp(min=-100)))
        b = v.view(rows, -1, 16)
        scale = (b.abs().amax(2) / (6 * row[:, None])).to(torch.float8_e4m3fn).float()
        unit = (scale * row[:, None])[:, :, None]
        q = torch.where(unit == 0, 0, _e2m1(b / torch.where(unit == 0, 1, unit)))
        return q.view(rows, width), scale, row
    b = v.view(rows, -1, 32)
    amax = b.abs().amax(2)
    e = torch.where(amax == 0, -127, _exponent(amax, fmt)).clamp(min=-127)
    t = b * _pow2(-e)[:, :, None]
    q = t.to(torch.float8_e4m3fn) if fmt == "mxe4m3" else _e2m1(t)
    return q.view(rows, width), _pow2(e), None


def _tile(scale, fill):
    """Block scales in the order the product reads them: blocks of 128 rows x 4 scales, the
    scale of row r, column c at (r % 32, r / 32, c)."""
    rows, cols = scale.shape
    s = torch.nn.functional.pad(scale, (0, _up(cols, 4) - cols, 0, _up(rows, 128) - rows), value=fill)
    return s.view(-1, 4, 32, s.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untile(tiled, rows, cols):
    s = tiled.view(_up(rows, 128) // 128, _up(cols, 4) // 4, 32, 4, 4).permute(0, 3, 2, 1, 4)
    return s.reshape(_up(rows, 128), _up(cols, 4))[:rows, :cols]


def _values(v, fmt):
    """What v's quantised rows stand for, without their padding."""
    q, scale, row = _split(v.float(), fmt)
    q = q.float()
    if scale is not None:
        q = q * scale.repeat_interleave(q.shape[1] // scale.shape[1], 1)
    return (q if row is None else q * row[:, None])[:, : v.shape[1]]


def _packed(v, fmt):
    """A 4-bit operand as it is kept: two codes a byte (the first one low), tiled scale
    bytes, row scales."""
    q, scale, row = _split(v.float(), fmt)
    a = q.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code += 8 * torch.signbit(q).to(torch.uint8)
    data = code[:, 0::2] + 16 * code[:, 1::2]
    if fmt == "nvfp4":
        scales = _tile(scale, 0.0).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        scales = _tile(torch.frexp(scale)[1].float() + 126, 0.0).to(torch.uint8)  # (the exponent's byte)
    return {"data": data.contiguous(), "scales": scales.contiguous(), "row_scale": row, "format": fmt,
            "cols": v.shape[1]}


def _unpacked(p, to):
    """What a kept 4-bit operand stands for."""
    data, fmt = p["data"], p["format"]
    rows, width = data.shape[0], 2 * data.shape[1]
    code = torch.stack([data & 15, data >> 4], 2).view(rows, width).int()
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=to, device=data.device)
    per = 16 if fmt == "nvfp4" else 32
    s = _untile(p["scales"], rows, width // per)
    s = s.view(torch.float8_e4m3fn).to(to) if fmt == "nvfp4" else _pow2(s.int() - 127).to(to)
    v = table[code] * s.repeat_interleave(per, 1)
    return (v if p["row_scale"] is None else v * p["row_scale"].to(to)[:, None])[:, : p["cols"]]


# ------------------------------------------------------------------------ inputs


def _make(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    c = case

    def normal(*shape, std=1.0, mean=0.0, to=torch.bfloat16):
        v = torch.randn(shape, generator=g, device="cuda")
        return v.mul_(std).add_(mean).to(to)

    def activations(rows, cols, to):
        v = torch.randn(rows, cols, generator=g, device="cuda")
        v[:, :: max(1, cols // 7)] *= 8  # a few large channels
        return v.to(to)

    if c["op"] == "quantise":
        return {"x": activations(c["rows"], c["cols"], DT[c["dtype"]])}
    if c["op"] == "norm":
        dt = DT[c["dtype"]]
        s = {"y": normal(c["M"], c["D"], std=1.5, mean=0.25, to=dt), "residual": normal(c["M"], c["D"], std=3.0, to=dt),
             "weight": normal(c["D"], std=0.2, mean=1.0, to=DT[c["param"]])}
        s["residual"][:, :: max(1, c["D"] // 7)] *= 8
        return s
    M, N, K = c["M"], c["N"], c["K"]
    std = 0.02 * math.sqrt(4096 / K)
    if c["op"] == "grad":
        dt = DT[c["dtype"]]
        return {"dy": normal(M, N, std=0.05, to=dt), "x": activations(M, K, dt), "w": normal(N, K, std=std, to=dt)}
    s = {"b": _packed(normal(N, K, std=std), c["format"])}
    if c["op"] == "product":
        s["a"] = _packed(activations(M, K, torch.bfloat16), c["format"])
        return s
    s["x"] = activations(M, K, DT[c["dtype"]])
    s["bias"] = normal(N, std=0.5, to=torch.float32) if c["fused"] else None
    s["residual"] = normal(M, N, std=2.0, to=DT[c["out"]]) if c["fused"] else None
    return s


def prepare(case, seed):
    return dict(_make(case, seed), case=case)


# ------------------------------------------------------------------- plain forms


def _act(name, g):
    if name == "relu":
        return g * (g > 0).float()
    if name == "silu":
        return g / (1 + torch.exp(-g))
    if name == "gelu_tanh":
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
    return g


def _plain_quantise(v, fmt):
    q, scale, row = _split(v, fmt)
    # (an empty place in the tiled scales holds the byte 0, which stands for 2^-127)
    return q, row if scale is None else _tile(scale, 2.0 ** -127).to(torch.float8_e8m0fnu)


def _plain(s, c):
    if c["op"] == "quantise":
        v = s["x"].float()
        return _plain_quantise(v.t() if c["transpose"] else v, c["format"])
    if c["op"] == "norm":
        t = s["residual"].float() + s["y"].float()
        n = t * torch.rsqrt(t.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
        return (t.to(s["y"].dtype),) + _plain_quantise(n, c["format"])
    if c["op"] == "grad":
        f = c["format"]
        dx = _values(s["dy"], f) @ _values(s["w"].t(), f).t()
        dw = _values(s["dy"].t(), f) @ _values(s["x"].t(), f).t()
        return dx.to(torch.bfloat16), dw.to(torch.bfloat16)
    a = _unpacked(s["a"], torch.float32) if c["op"] == "product" else _values(s["x"], c["format"])
    y = a @ _unpacked(s["b"], torch.float32).t()
    if c["op"] == "linear":
        y = _act(c["act"], y if s["bias"] is None else y + s["bias"])
        y = y if s["residual"] is None else y + s["residual"].float()
    return y.to(DT[c["out"]])


def run(state):
    c = state["case"]
    if not own:
        return _plain(state, c)
    from dense_gemm_blackwell_sm_gb300 import quant

    if c["op"] == "quantise":
        q = quant.quantise(state["x"], c["format"], transpose=c["transpose"])
        return q.data, q.row_scale if q.scales is None else q.scales.view(torch.float8_e8m0fnu)
    if c["op"] == "norm":
        t, q = quant.norm_quantise(state["y"], state["residual"], state["weight"], format=c["format"], eps=EPS)
        return t, q.data, q.row_scale if q.scales is None else q.scales.view(torch.float8_e8m0fnu)
    if c["op"] == "grad":
        return quant.linear_backward(state["dy"], state["x"], state["w"], format=c["format"])
    b = quant.Quantised(**state["b"])
    if c["op"] == "product":
        return quant.product(quant.Quantised(**state["a"]), b, static_b=True)
    return quant.linear(state["x"], b, bias=state["bias"], act=c["act"], residual=state["residual"],
                        out_dtype=DT[c["out"]], static_b=True)


# ------------------------------------------------- the definitions in 64 bits

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nearest4(t):
    """The nearest 4-bit value of t: how many midpoints lie below it, a tie taking the even code."""
    a = t.abs()
    index = torch.zeros_like(a)
    for code in range(1, 8):
        mid = (GRID[code - 1] + GRID[code]) / 2
        index += (a > mid) if code % 2 else (a >= mid)
    return torch.tensor(GRID, dtype=t.dtype, device=t.device)[index.int()] * torch.where(torch.signbit(t), -1.0, 1.0)


def _two_to(e):
    """2^e in 64 bits, for a whole number e, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest8(t):
    """The nearest E4M3 value: 3 bits behind the leading one, steps of 2^-9 below 2^-6."""
    e = torch.round(torch.log2(t.abs().clamp(min=2.0 ** -6)))
    e = torch.where((t.abs() < _two_to(e)) & (e > -6), e - 1, e)
    step = _two_to(e - 3)
    return (torch.round(t / step) * step).clamp(-448, 448)


def _covering(amax, largest):
    """The smallest whole e with amax <= largest * 2^e (0 for amax 0)."""
    e = torch.round(torch.log2(torch.where(amax > 0, amax, largest) / largest))
    e = torch.where(amax > largest * _two_to(e), e + 1, e)
    return torch.where((amax > 0) & (amax <= largest * _two_to(e - 1)), e - 1, e)


def _exact_split(v, fmt):
    """Values and scales of v's rows (64 bits), blocks as the last axis."""
    per = {"e4m3": 0, "mxe4m3": 32, "mxfp4": 32, "nvfp4": 16}[fmt]
    rows, cols = v.shape
    pad = torch.zeros(rows, max(32, _up(cols, 32)) - cols, dtype=v.dtype, device=v.device)
    v = torch.cat([v, pad], 1)
    top = v.abs().max(1, keepdim=True).values
    if fmt == "e4m3":
        scale = (top / 448).clamp(min=2.0 ** -126)
        return _nearest8(v / scale), None, scale[:, 0]
    b = v.reshape(rows, -1, per)
    most = b.abs().max(2).values
    if fmt == "nvfp4":
        row = torch.where(top > 0, _two_to(_covering(top, 2688.0).clamp(min=-100)), 1.0)
        scale = _nearest8(most / (6 * row))
        unit = scale * row
        q = torch.where(unit[:, :, None] > 0, _nearest4(b / unit[:, :, None]), 0.0)
        return q.reshape(v.shape), scale, row[:, 0]
    scale = _two_to(torch.where(most > 0, _covering(most, 448.0 if fmt == "mxe4m3" else 6.0), -127.0).clamp(min=-127))
    q = (_nearest8 if fmt == "mxe4m3" else _nearest4)(b / scale[:, :, None])
    return q.reshape(v.shape), scale, None


def _exact_values(v, fmt):
    q, scale, row = _exact_split(v, fmt)
    q = (q.view(q.shape[0], scale.shape[1], -1) * scale[:, :, None]).reshape(q.shape)
    return (q if row is None else q * row[:, None])[:, : v.shape[1]]


def _exact_quantised(v, fmt):
    q, scale, row = _exact_split(v, fmt)
    if scale is None:
        return q, row
    rows, cols = scale.shape
    tiled = torch.full((_up(rows, 128), _up(cols, 4)), 2.0 ** -127, dtype=v.dtype, device=v.device)
    tiled[:rows, :cols] = scale
    return q, torch.cat([torch.stack(band.view(4, 32, -1, 4).unbind(0), 2)[:, k].reshape(-1)
                         for band in tiled.split(128) for k in range(tiled.shape[1] // 4)])


def _exact_act(name, g):
    if name == "relu":
        return torch.clamp(g, min=0)
    if name == "silu":
        return g * torch.sigmoid(g)
    if name == "gelu_tanh":
        return g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
    return g


def exact(case, seed):
    c = case
    s = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in _make(case, seed).items()}
    if c["op"] == "quantise":
        return _exact_quantised(s["x"].t() if c["transpose"] else s["x"], c["format"])
    if c["op"] == "norm":
        t = s["y"] + s["residual"]
        n = t / torch.sqrt((t * t).sum(1, keepdim=True) / c["D"] + EPS) * s["weight"]
        return (t,) + _exact_quantised(n, c["format"])
    if c["op"] == "grad":
        f = c["format"]
        dx = _exact_values(s["dy"], f) @ _exact_values(s["w"].t(), f).t()
        return dx, _exact_values(s["dy"].t(), f) @ _exact_values(s["x"].t(), f).t()
    a = _unpacked(s["a"], torch.float64) if c["op"] == "product" else _exact_values(s["x"], c["format"])
    y = a @ _unpacked(s["b"], torch.float64).t()
    if c["op"] == "linear":
        y = _exact_act(c["act"], y if s["bias"] is None else y + s["bias"])
        y = y if s["residual"] is None else y + s["residual"]
    return y
