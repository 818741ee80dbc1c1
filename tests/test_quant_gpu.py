"""Quantisation by rows and by columns, and the norm with a quantised output, against their
definitions in 64 bits: codes and scales of a given input bit for bit, what follows a norm
within the bounds of its fp32 arithmetic and half a step of the format."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import ffn as bounds
from oracle import quant as ref
from dense_gemm_blackwell_sm_gb300 import ffn, gemm, quant

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FORMATS = ["e4m3", "mxe4m3", "mxfp4", "nvfp4"]
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def f64(t):
    return t.double().cpu().numpy()


def inputs(rows, cols, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(spread * torch.randn(rows, 1, generator=g))
    if cols > 8:
        x[:, 5] *= 20
    return x.to(DT[dtype])


def check_operand(q, want):
    """A Quantised's bytes against the oracle's Operand."""
    rows = want.codes.shape[0]
    data = q.data.view(torch.uint8).cpu().numpy()
    codes = want.codes if q.format in ("e4m3", "mxe4m3") else ref.packed(want.codes)
    bad = np.argwhere(data != codes)
    assert data.shape == codes.shape and bad.size == 0, (len(bad), bad[:4])
    if want.scales is None:
        assert q.scales is None
    else:
        got, tiled = q.scales.cpu().numpy(), ref.tile(want.scales, rows)
        bad = np.argwhere(got != tiled)
        assert got.shape == tiled.shape and bad.size == 0, (len(bad), bad[:4])
    if want.row_scale is None:
        assert q.row_scale is None
    else:
        assert np.array_equal(f64(q.row_scale), want.row_scale, equal_nan=True)


# one element; one block; odd widths; several blocks; a warp's, a CTA's and more than a CTA's row
SHAPES = [(1, 1), (1, 32), (3, 31), (5, 33), (7, 1001), (130, 512), (2, 4096), (300, 96), (2, 16384), (1, 40000)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rows(shape, fmt, dtype):
    x = inputs(*shape, dtype, seed=sum(shape))
    q = quant.quantise(x.to(DEV), fmt)
    assert quant.check() == gemm.OK
    assert q.format == fmt and q.cols == shape[1]
    check_operand(q, ref.quantise(f64(x), fmt))


@pytest.mark.parametrize("shape", [(1, 1), (31, 3), (32, 64), (33, 65), (1001, 7), (512, 130), (257, 200), (40, 1),
                                   (3000, 70)])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_columns(shape, fmt, dtype):
    x = inputs(*shape, dtype, seed=sum(shape))
    q = quant.quantise(x.to(DEV), fmt, transpose=True)
    assert quant.check() == gemm.OK
    assert q.cols == shape[0]
    check_operand(q, ref.quantise(f64(x).T, fmt))


@pytest.mark.parametrize("fmt", FORMATS)
def test_ties_zeros_and_extremes(fmt):
    # every midpoint of both formats under several scales, zeros of both signs, subnormals, the
    # largest values of the types
    mids = np.concatenate([(ref.E2M1[1:8] + ref.E2M1[:7]) / 2, (ref.E4M3[1:127] + ref.E4M3[:126]) / 2])
    rows = []
    for s in (1.0, 1.125, 1.25, 1.375, 1.5, 1.625, 1.75, 1.875, 2.0 ** -20):
        r = np.zeros(256)
        for i, m in enumerate(mids[:224]):
            r[i // 14 * 16 + i % 14] = m * s * (-1) ** i
        r[14::16] = 6.0 * s   # a block's largest value makes NVFP4's scale s, times a power of two
        r[15] = 2688.0
        rows.append(r)
    x = torch.tensor(np.array(rows), dtype=torch.float32)
    extra = torch.zeros(6, 256)
    extra[1] = -0.0
    extra[2, :7] = torch.tensor([1e-40, -1e-45, 3e-39, 0, 1e-38, 2.0 ** -149, 2.0 ** -126])
    extra[3, 17], extra[3, 100] = torch.finfo(torch.float32).max, -1.0
    extra[4, 3] = 2.0 ** -100
    extra[5, :32] = 2.0 ** -130
    for t in (x, x.bfloat16().float(), extra):
        check_operand(quant.quantise(t.to(DEV), fmt), ref.quantise(f64(t), fmt))
        check_operand(quant.quantise(t.t().contiguous().to(DEV), fmt, transpose=True), ref.quantise(f64(t), fmt))
    for dt in (torch.bfloat16, torch.float16):
        t = x.clamp(-60000, 60000).to(dt)
        check_operand(quant.quantise(t.to(DEV), fmt), ref.quantise(f64(t), fmt))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("transpose", [False, True])
def test_rows_of_nan_and_infinity(fmt, transpose):
    x = inputs(140, 200, "bf16", 3)
    x[0, 7], x[65, 199], x[130, 0] = float("nan"), float("inf"), -float("inf")
    t = x.t().contiguous() if transpose else x
    check_operand(quant.quantise(t.to(DEV), fmt, transpose=transpose), ref.quantise(f64(x), fmt))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("offset,pitch", [(0, 104), (8, 104), (1, 101), (3, 160)])
def test_strided_rows(fmt, transpose, offset, pitch):
    # rows inside a wider array, on and off 16-byte boundaries
    base = inputs(90, pitch, "f16", 11).to(DEV)
    x = base[:, offset:offset + 97]
    got = quant.quantise(x, fmt, transpose=transpose)
    check_operand(got, ref.quantise(f64(x).T if transpose else f64(x), fmt))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape,transpose", [((0, 40), False), ((5, 0), False), ((0, 5), True), ((40, 0), True)])
def test_nothing(fmt, shape, transpose):
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    q = quant.quantise(x, fmt, transpose=transpose)
    rows, cols = shape[::-1] if transpose else shape
    assert q.cols == cols and q.data.shape[0] == rows
    check_operand(q, ref.quantise(np.zeros((rows, cols)), fmt))


def test_past_two_to_the_31_elements():
    # offsets of the last rows pass 2^31: compared with the same rows alone
    rows, cols = 66000, 32800
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    x.zero_()
    tail = inputs(64, cols, "bf16", 5).to(DEV)
    x[-64:] = tail
    for fmt in ("mxfp4", "nvfp4"):
        q, alone = quant.quantise(x, fmt), quant.quantise(tail, fmt)
        assert torch.equal(q.data[-64:], alone.data)
        if fmt == "nvfp4":
            assert torch.equal(q.row_scale[-64:], alone.row_scale)
        del q
    tall = x.view(-1, 32)[:, :4]  # its columns are rows of more than 2^26 elements
    first = (tall.shape[0] - 65600 + 31) // 32 * 32  # a block's first
    q, alone = (quant.quantise(t, "mxfp4", transpose=True) for t in (tall, tall[first:]))
    assert torch.equal(q.data[:, first // 2:], alone.data)


# ------------------------------------------------------------------------------ norm


def check_norm(q, n, en, dtype):
    """Codes of values known to within en: the scales follow the rule for the largest value within its
    bound, each value is within half a step of its code, or as far as a limited one is."""
    rows, cols = n.shape
    w = ref.width(cols)
    if q.format in ("e4m3", "mxe4m3"):
        codes, table = q.data.view(torch.uint8).cpu().numpy(), ref.E4M3
    else:
        b = q.data.cpu().numpy()
        codes, table = np.stack([b & 15, b >> 4], 2).reshape(rows, w), ref.E2M1
    v, ev = np.zeros((rows, w)), np.zeros((rows, w))
    v[:, :cols], ev[:, :cols] = n, en
    o = ref.Operand(codes, None, None, q.format, cols)
    if q.row_scale is not None:
        o = o._replace(row_scale=f64(q.row_scale))
    if q.scales is not None:
        per = ref.BLOCK[q.format]
        where = ref.tile(np.arange(256).astype(np.uint8)[None, :0], 0)  # (empty: shapes only)
        assert where.size == 0
        sc = w // per
        flat = q.scales.cpu().numpy()
        r, c = np.meshgrid(np.arange(rows), np.arange(sc), indexing="ij")
        cb = -(-sc // 4)
        at = ((r // 128) * cb + c // 4) * 512 + (r % 32) * 16 + ((r // 32) % 4) * 4 + c % 4
        o = o._replace(scales=flat[at])
        assert np.array_equal(ref.tile(o.scales, rows), flat)  # (and zeros elsewhere)
    top = np.abs(v).max(1)
    etop = (ev.max(1) + 4 * bounds.E * top)
    if q.format == "e4m3":
        assert (np.abs(o.row_scale - np.maximum(top / 448, 2.0 ** -126)) <= etop / 448 + 4 * bounds.E * o.row_scale).all()
    elif q.format == "nvfp4":
        low, high = (ref.covering(np.maximum(top + s * etop, 1e-30), 2688.0) for s in (-1, 1))
        k = np.log2(o.row_scale)
        assert ((top == 0) | ((k >= low) & (k <= high))).all()
        b = np.abs(v).reshape(rows, -1, 16).max(2)
        eb = ev.reshape(rows, -1, 16).max(2) + 4 * bounds.E * b
        s = [ref.E4M3[ref.e4m3(np.maximum(b + d * eb, 0) / (6 * o.row_scale[:, None]))] for d in (-1, 1)]
        got = ref.E4M3[o.scales]
        assert ((got >= s[0]) & (got <= s[1])).all()
    else:
        b = np.abs(v).reshape(rows, -1, 32).max(2)
        eb = ev.reshape(rows, -1, 32).max(2) + 4 * bounds.E * b
        low, high = (ref.covering(np.maximum(b + s * eb, 1e-30), ref.LARGEST[q.format]) for s in (-1, 1))
        e = o.scales.astype(int) - 127
        assert ((b == 0) | ((e >= low) & (e <= high))).all()
    unit = ref.unit(o)
    got = table[codes] * unit
    step = ref.half_step(codes, table) * unit
    limited = np.abs(table[codes]) == (6.0 if table is ref.E2M1 else 448.0)
    extra = np.where(limited, np.abs(v) / 16, 0) if q.format == "nvfp4" else 0
    assert (np.abs(got - v) <= step + ev + 4 * bounds.E * np.abs(v) + extra).all()


@pytest.mark.parametrize("shape", [(1, 1), (1, 4096), (5, 33), (130, 512), (257, 1000), (3, 8192), (2, 32768), (40, 1001)])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_norm(shape, fmt, dtype):
    y, res = inputs(*shape, dtype, 1, 0.3), inputs(*shape, dtype, 2, 0.3)
    weight = 1 + 0.2 * torch.randn(shape[1], generator=torch.Generator().manual_seed(3))
    if shape[1] % 2:
        weight = weight.to(DT[dtype])
    s, q = quant.norm_quantise(y.to(DEV), res.to(DEV), weight.to(DEV), format=fmt, eps=1e-6, residual_scale=0.75,
                               branch_scale=1.5)
    assert quant.check() == gemm.OK
    want, (n, en) = ref.norm(f64(y), f64(res), f64(weight), dtype, 1e-6, 0.75, 1.5)
    bad, worst = bounds.outside(f64(s), want)
    assert bad == 0, (bad, worst)
    check_norm(q, n, en, dtype)


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4"])
def test_norm_without_parts_and_in_place(fmt):
    y, res = inputs(20, 96, "bf16", 1), inputs(20, 96, "bf16", 2)
    none, q = quant.norm_quantise(y.to(DEV), format=fmt, need_s=False)
    assert none is None
    _, (n, en) = ref.norm(f64(y), None, None, "bf16", 1e-6)
    check_norm(q, n, en, "bf16")
    s0, q0 = quant.norm_quantise(y.to(DEV), res.to(DEV), format=fmt)
    for place in ("residual", "y"):
        a, b = y.to(DEV), res.to(DEV)
        s, q = quant.norm_quantise(a, b, format=fmt, s=b if place == "residual" else a)
        assert s.data_ptr() == (b if place == "residual" else a).data_ptr()
        assert torch.equal(s, s0) and torch.equal(q.data.view(torch.uint8), q0.data.view(torch.uint8))
    zero = torch.zeros(3, 64, dtype=torch.bfloat16, device=DEV)
    s, q = quant.norm_quantise(zero, format=fmt)
    assert not s.any() and not q.data.view(torch.uint8).any()
    s, q = quant.norm_quantise(zero[:0], format=fmt)
    assert s.shape == (0, 64) and q.data.shape[0] == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_norm_strided_and_nan(fmt):
    base, rbase = inputs(40, 101, "f16", 1).to(DEV), inputs(40, 99, "f16", 2).to(DEV)
    y, res = base[:, 2:99], rbase[:, 1:98]
    s, q = quant.norm_quantise(y, res, format=fmt)
    want, (n, en) = ref.norm(f64(y), f64(res), None, "f16", 1e-6)
    assert bounds.outside(f64(s), want)[0] == 0
    check_norm(q, n, en, "f16")
    y = inputs(4, 64, "bf16", 3).to(DEV)
    y[1, 5], y[2, 6] = float("nan"), float("inf")
    _, q = quant.norm_quantise(y, format=fmt)
    for r in (1, 2):
        if q.row_scale is not None:
            assert torch.isnan(q.row_scale[r])
        else:
            sc = q.scales.view(-1, 512)  # (an infinity leaves 0 in the row's other block)
            assert (sc[:, 16 * r:16 * r + 2] == 255).any() and not (sc[:, 0] == 255).any()


def test_norm_is_block_norm_s():
    # the same s bit for bit as the unquantised operator, whose gradient is this one's
    y, res = inputs(64, 256, "bf16", 1).to(DEV), inputs(64, 256, "bf16", 2).to(DEV)
    w = (1 + 0.1 * torch.randn(256, generator=torch.Generator().manual_seed(1))).to(DEV)
    s, n = ffn.block_norm(y, res, pre_weight=w)
    s2, q = quant.norm_quantise(y, res, w, format="e4m3")
    assert torch.equal(s, s2)
    back = q.data.float() * q.row_scale[:, None]
    # half a step of E4M3 is 2^-4 of the value (2^-10 of the scale below its normal range), and n is rounded to bf16
    err, room = (back - n.float()).abs(), n.float().abs() * (2.0 ** -4 + 2.0 ** -7) + q.row_scale[:, None] * 2.0 ** -9
    assert (err <= room).all()


# ---------------------------------------------------------------- streams and graphs


@pytest.mark.parametrize("transpose", [False, True])
def test_other_stream_and_graph(transpose):
    x = inputs(300, 520, "bf16", 9).to(DEV)
    want = quant.quantise(x, "nvfp4", transpose=transpose)
    side = torch.cuda.Stream()
    got = quant.quantise(x, "nvfp4", transpose=transpose, stream=side)
    side.synchronize()
    assert torch.equal(got.data, want.data) and torch.equal(got.scales, want.scales)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = quant.quantise(x, "nvfp4", transpose=transpose)
    other = inputs(300, 520, "bf16", 10).to(DEV)
    want = quant.quantise(other, "nvfp4", transpose=transpose)
    x.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept.data, want.data) and torch.equal(kept.row_scale, want.row_scale)


def test_refusals_of_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        quant.quantise(x, "fp4")
    with pytest.raises(ValueError):
        quant.quantise(x.double(), "e4m3")
    with pytest.raises(ValueError):
        quant.quantise(x.t(), "e4m3")
    with pytest.raises(ValueError):
        quant.quantise(x[0], "e4m3")
    with pytest.raises(ValueError):
        quant.norm_quantise(x, x[:2], format="e4m3")
    with pytest.raises(ValueError):
        quant.norm_quantise(x, weight=torch.ones(63, device=DEV), format="e4m3")
    with pytest.raises(ValueError):
        quant.norm_quantise(x, weight=torch.ones(64, device=DEV, dtype=torch.float16), format="e4m3")
    with pytest.raises(gemm.GemmError):
        quant.norm_quantise(torch.zeros(1, 32769, dtype=torch.bfloat16, device=DEV), format="e4m3")


# columns with a scale each: one part and many, of unequal length; few columns and many, ragged and
# off a boundary
WHOLE = [(1, 3), (64, 65), (130, 70), (512, 20000), (1000, 513), (1025, 100), (2049, 64), (4097, 260), (8193, 40), (14336, 33),
         (14337, 33), (20000, 70)]


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4"])
@pytest.mark.parametrize("shape", WHOLE)
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_columns_are_the_rows_of_the_transpose(fmt, shape, dtype):
    # (rows are compared with the definition above; columns may differ from them in no bit)
    gen = torch.Generator().manual_seed(shape[0])
    wide = torch.randn(shape[0], shape[1] + 9, generator=gen) * 2.0 ** torch.randint(-4, 5, (1, shape[1] + 9), generator=gen)
    wide[shape[0] // 2, 1:shape[1]:7] = 0
    wide[:, 2::11] = 0
    wide[shape[0] - 1, 5::13] = float("nan")
    wide = wide.to(DEV, dtype)
    for x in (wide[:, :shape[1]].contiguous(), wide[:, 3:shape[1] + 3]):
        got, want = quant.quantise(x, fmt, transpose=True), quant.quantise(x.t().contiguous(), fmt)
        for a, b in ((got.data, want.data), (got.scales, want.scales), (got.row_scale, want.row_scale)):
            assert (a is None and b is None) or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("transpose", [False, True])
def test_fp32_values_beside_every_tie_of_nvfp4(transpose):
    # every scale s, every midpoint b of the codes: b s and the floats beside it, in blocks whose
    # largest value is 6 s; then every midpoint of the scales, and beside it, as a block's largest value.
    # One block holds 2688, so that the row's scale is one.
    e4m3 = ref.E4M3[1:127]
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    blocks = [np.full(16, 2688.0, np.float32)]
    for s in e4m3:
        ties = (mids * s).astype(np.float32)
        v = np.concatenate([ties, np.nextafter(ties, np.float32(np.inf)), -np.nextafter(ties, np.float32(0))])
        for part in (v[:15], np.concatenate([v[15:], v[:9]])):
            blocks.append(np.concatenate([[np.float32(6 * s)], part]).astype(np.float32))
    middle = ((e4m3[1:] + e4m3[:-1]) / 2 * 6).astype(np.float32)
    for m in np.concatenate([middle, np.nextafter(middle, np.float32(np.inf)), np.nextafter(middle, np.float32(0))]):
        blocks.append(np.concatenate([[m], np.linspace(-1, 1, 15) * m]).astype(np.float32))
    x = np.stack([np.concatenate(blocks), -np.concatenate(blocks)])
    assert (np.abs(x).max(1) == 2688).all()
    t = torch.tensor(x, device=DEV)
    got = quant.quantise(t.t().contiguous() if transpose else t, "nvfp4", transpose=transpose)
    want = ref.quantise(x.astype(np.float64), "nvfp4")
    assert (want.row_scale == 1).all()
    check_operand(got, want)
