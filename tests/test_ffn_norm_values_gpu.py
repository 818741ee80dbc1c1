"""The block norms with parameters that are not finite: what a row holds past its ends
does not come into its sums."""
from __future__ import annotations

import pytest
import torch

from dense_gemm_blackwell_sm_gb300 import ffn, gemm
from test_ffn_gpu import DEV, norm_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert ffn.check() == gemm.OK


@pytest.mark.parametrize("M", [6, 5000])
@pytest.mark.parametrize("D,column", [(255, 254), (255, 0), (256, 255), (907, 906)])
@pytest.mark.parametrize("which", ["post_weight", "gate"])
def test_an_infinite_factor_at_a_rows_end(M, D, column, which):
    """s is infinite in that column, so the RMS is, and the other columns of n are zero: nothing of
    the places past a row's end comes in."""
    t, p = norm_inputs(M, D, "bf16", "f32", "rms", 1, D)
    p[which][..., column] = float("inf")
    s, n = ffn.block_norm(t["y"], t["residual"], post_norm=True, **p)
    others = torch.arange(D, device=DEV) != column
    y_there = t["y"][:, column] != 0  # (zero times infinity is NaN)
    assert bool(s[y_there, column].isinf().all()) and bool(s[:, others].isfinite().all())
    assert bool((n[y_there][:, others] == 0).all()) and bool(n[:, column].isnan().all())


@pytest.mark.parametrize("M", [6, 5000])
@pytest.mark.parametrize("D", [255, 256])
def test_an_infinite_gate_without_a_bias(M, D):
    t, p = norm_inputs(M, D, "bf16", "f32", "layer", 1, D)
    p["post_bias"] = None
    p["gate"][..., 3] = float("inf")
    s, _ = ffn.block_norm(t["y"], t["residual"], post_norm=True, kind="layer", **p)
    assert bool(s[:, 3].isinf().all()) and bool(s[:, 4:].isfinite().all())


@pytest.mark.parametrize("M", [6, 2000])
@pytest.mark.parametrize("D,column", [(255, 254), (256, 255), (1031, 1030), (5001, 5000)])
def test_gradient_with_an_infinite_factor_at_a_rows_end(M, D, column):
    """dz is infinite in that column, so mean(b v) is, and the other columns of dy with it (RMS)."""
    t, p = norm_inputs(M, D, "bf16", "f32", "rms", 1, D)
    s, _ = ffn.block_norm(t["y"], t["residual"], post_norm=True, **p)
    p["gate"][..., column] = float("inf")
    got = ffn.block_norm_backward(t["ds"], t["dn"], t["y"], s, post_norm=True, **p)
    others = (torch.arange(D, device=DEV) != column) & (t["y"] != 0).all(0)
    there = (t["y"][:, column] != 0) & (got.dresidual[:, column] != 0)
    assert bool(got.dy[there][:, others].isinf().all())
    assert bool(got.dresidual.isfinite().all())
