"""The block norms at the end of their range of widths, rows that are no multiple of 16
bytes and rows off their boundary among them, against the 64-bit definitions."""
from __future__ import annotations

import pytest
import torch

from dense_gemm_blackwell_sm_gb300 import ffn, gemm
from test_ffn_gpu import DEV, assert_within, norm_inputs, ref_norm, ref_norm_grad

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert ffn.check() == gemm.OK


def rows_at(v, off, pitch):
    """A copy of v whose rows lie `pitch` apart, `off` elements past a boundary, amid NaN."""
    M, D = v.shape
    flat = torch.full((off + M * pitch + 16,), float("nan"), dtype=v.dtype, device=DEV)
    view = flat[off:off + M * pitch].view(M, pitch)[:, :D]
    view.copy_(v)
    return view


# the widths where a thread count of either direction was once too large, and their neighbours
WIDE = [32640, 32641, 32648, 32650, 32704, 32761, 32762, 32765, 32766, 32767, 32768]
OFF = [(1, 0), (0, 1), (3, 5)]  # elements past a boundary, elements between rows


def check_forward(t, p, dtype, kind):
    s, n = ffn.block_norm(t["y"], t["residual"], post_norm=True, kind=kind, **p)
    want_s, want_n = ref_norm(t, p, dtype, post=True, pre=True, kind=kind, eps=1e-6)
    assert_within(s, want_s, "s")
    assert_within(n, want_n, "n")


@pytest.mark.parametrize("D", WIDE)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_widest_rows(D, dtype, kind):
    t, p = norm_inputs(3, D, dtype, "f32", kind, 1, D)
    check_forward(t, p, dtype, kind)


@pytest.mark.parametrize("D", [32762, 32767, 32768])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("off,gap", OFF)
def test_widest_rows_off_their_boundary(D, dtype, off, gap):
    t, p = norm_inputs(3, D, dtype, "f32", "rms", 1, D)
    check_forward({k: rows_at(v, off, D + gap) for k, v in t.items()}, p, dtype, "rms")


def test_widest_rows_for_a_prompt():
    t, p = norm_inputs(400, 32767, "bf16", "bf16", "layer", 4, 5)
    check_forward(t, p, "bf16", "layer")


def check_gradient(t, p, dtype, kind):
    s, _ = ffn.block_norm(t["y"], t["residual"], post_norm=True, kind=kind, **p)
    got = ffn.block_norm_backward(t["ds"], t["dn"], t["y"], s, post_norm=True, kind=kind, **p)
    want = ref_norm_grad(t, p, s, dtype, post=True, pre=True, kind=kind, eps=1e-6)
    for name, g, b in zip(got._fields, got, want):
        assert (g is None) == (b is None), name
        if g is not None:
            assert_within(g, b, name)


@pytest.mark.parametrize("D", WIDE)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_widest_gradients(D, dtype, kind):
    t, p = norm_inputs(3, D, dtype, "f32", kind, 1, D)
    check_gradient(t, p, dtype, kind)


@pytest.mark.parametrize("D", [32641, 32767, 32768])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("off,gap", OFF)
def test_widest_gradients_off_their_boundary(D, dtype, off, gap):
    t, p = norm_inputs(3, D, dtype, "f32", "rms", 1, D)
    check_gradient({k: rows_at(v, off, D + gap) for k, v in t.items()}, p, dtype, "rms")


@pytest.mark.parametrize("D", [32641, 32767])
def test_widest_gradients_with_gates(D):
    """A gate for few rows (whole groups per part), and few gates over many rows."""
    t, p = norm_inputs(6, D, "bf16", "f32", "layer", 3, D)
    check_gradient(t, p, "bf16", "layer")
    t, p = norm_inputs(600, D, "bf16", "bf16", "rms", 2, D)
    check_gradient(t, p, "bf16", "rms")
