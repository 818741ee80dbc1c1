"""The oracle of the low-precision operands, pinned: format tables, ties, brute force over
all candidates, scale rules by their own definition, and planted mistakes that must show."""
from __future__ import annotations

import itertools

import numpy as np
import pytest
import torch

from oracle import quant as ref

FORMATS = ["e4m3", "mxe4m3", "mxfp4", "nvfp4"]


def test_e4m3_table_is_torch_s():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(ref.E4M3))
    fine = ~np.isnan(t)
    assert np.array_equal(t[fine], ref.E4M3[fine]) and np.array_equal(np.signbit(t[fine]), np.signbit(ref.E4M3[fine]))


@pytest.mark.parametrize("table,code", [(ref.E2M1[:8], ref.e2m1), (ref.E4M3[:127], ref.e4m3)])
def test_nearest_by_brute_force(table, code):
    rng = np.random.default_rng(0)
    mid = (table[1:] + table[:-1]) / 2
    t = np.concatenate([table, mid, mid * (1 + 2.0 ** -30), mid * (1 - 2.0 ** -30), rng.uniform(0, 1.2 * table[-1], 500)])
    for v in t:
        got = int(code(np.array([v]))[0])
        d = np.abs(table - v)
        best = [i for i in range(len(table)) if d[i] == d.min()]
        want = best[0] if len(best) == 1 else next(i for i in best if i % 2 == 0)
        assert got == want, (v, got, want)
        if v > 0:
            assert int(code(np.array([-v]))[0]) == want + (8 if len(table) == 8 else 128)


def test_e4m3_rounding_is_torch_s():
    x = np.random.default_rng(1).normal(size=4000) * 60
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3(x.astype(np.float64)), want)


@pytest.mark.parametrize("largest", [448.0, 6.0, 2688.0])
def test_covering_is_the_smallest_power(largest):
    rng = np.random.default_rng(2)
    a = np.concatenate([2.0 ** rng.uniform(-60, 60, 300), largest * 2.0 ** np.arange(-20, 20),
                        largest * 2.0 ** np.arange(-20, 20) * (1 + 2.0 ** -40)])
    e = ref.covering(a, largest)
    assert (a <= largest * 2.0 ** e).all() and (a > largest * 2.0 ** (e - 1)).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (5, 32), (4, 33), (2, 100), (130, 64)])
def test_quantise_holds_its_definition(fmt, rows, cols):
    rng = np.random.default_rng(rows * cols)
    x = (rng.normal(size=(rows, cols)) * np.exp(rng.normal(size=(rows, cols)))).astype(np.float32).astype(np.float64)
    x[0, : cols // 2] = 0
    o = ref.quantise(x, fmt)
    v = ref.values(o)
    assert v.shape == (rows, ref.width(cols)) and not v[:, cols:].any()
    table = ref.E2M1 if fmt in ("mxfp4", "nvfp4") else ref.E4M3
    unit = ref.unit(o)
    pad = np.zeros_like(v)
    pad[:, :cols] = x
    # within half a step of the code taken; NVFP4's scale is rounded, so its largest may be cut off
    step = ref.half_step(o.codes, table) * unit
    top = np.isin(np.abs(table[o.codes]), [6.0, 448.0])
    err = np.abs(v - pad)
    slack = 1e-6 * np.abs(pad)
    assert (err <= step + slack + (np.where(top, np.abs(pad) / 16, 0) if fmt == "nvfp4" else 0)).all()
    if fmt != "e4m3":
        assert ref.tile(o.scales, rows).size == -(-rows // 128) * -(-o.scales.shape[1] // 4) * 512


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_of_zeros_and_of_nothing_finite(fmt):
    x = np.zeros((4, 40))
    x[1, 3], x[2, 39] = np.nan, np.inf
    x[3] = 1.0
    o = ref.quantise(x, fmt)
    assert not ref.values(o)[0].any()
    with np.errstate(invalid="ignore"):
        s = ref.values(o).sum(1)
    assert np.isnan(s[1]) and np.isnan(s[2]) and np.isfinite(s[3])


def test_tile_order_is_mx_s():
    from dense_gemm_blackwell_sm_gb300 import inputs

    s = np.random.default_rng(3).integers(0, 255, (200, 11)).astype(np.uint8)
    want = inputs.mx_tile_scales(torch.tensor(s), 11 * 32).numpy()
    got = ref.tile(s, 200)
    r, c = np.meshgrid(np.arange(200), np.arange(11), indexing="ij")
    at = ((r // 128) * 3 + c // 4) * 512 + (r % 32) * 16 + ((r // 32) % 4) * 4 + c % 4
    assert got.size == want.size and np.array_equal(got[at], want[at])


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_product_of_all_codes(fmt):
    # every pair of codes once, scale 1: a sum of exact products by hand
    codes = np.array(list(itertools.product(range(16), range(16))), dtype=np.uint8)
    one = 56 if fmt == "nvfp4" else 127
    per = ref.BLOCK[fmt]
    a = ref.Operand(codes[:, 0].reshape(1, -1), np.full((1, 256 // per), one, np.uint8), None, fmt, 256)
    b = ref.Operand(codes[:, 1].reshape(1, -1), np.full((1, 256 // per), one, np.uint8), None, fmt, 256)
    v, bound = ref.product(a, b, "f32")
    assert v[0, 0] == sum(ref.E2M1[i] * ref.E2M1[j] for i, j in codes) and bound[0, 0] < 1e-2


@pytest.mark.parametrize("mistake", ["nibbles", "scale row", "tie"])
def test_planted_mistakes_show(mistake):
    rng = np.random.default_rng(4)
    x = rng.normal(size=(40, 64)).astype(np.float32).astype(np.float64)
    x[:, 0], x[:, 1] = 6.0, 2.5
    o = ref.quantise(x, "mxfp4")
    if mistake == "nibbles":
        assert not np.array_equal(ref.packed(o.codes), o.codes[:, 1::2] | (o.codes[:, 0::2] << 4))
    elif mistake == "scale row":
        assert not np.array_equal(ref.tile(o.scales, 40), ref.tile(np.roll(o.scales, 1, 0), 40))
    else:
        assert ref.E2M1[ref.e2m1(np.array([2.5, 0.25, 5.0]))].tolist() == [2.0, 0.0, 4.0]
