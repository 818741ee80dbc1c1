"""The norms' bounded waits: one that runs out (2 s) ends in a status, not in a hang, in
every form of the kernels, and the next call is whole."""
from __future__ import annotations

import ctypes

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


def missing(call, args):
    """The call with one arrival missing."""
    args.debug_flags = ffn.DEBUG_SKIP_ONE_LOAD
    assert call(ctypes.byref(args), torch.cuda.current_stream().cuda_stream) == gemm.OK
    assert ffn.check() == gemm.ERR_DEVICE_TIMEOUT
    assert ffn.check() == gemm.OK


# a warp per row, and a CTA
@pytest.mark.parametrize("M,D", [(5000, 200), (3000, 1031)])
def test_forward(M, D):
    t, p = norm_inputs(M, D, "bf16", "f32", "rms", 1, D)
    want = ffn.block_norm(t["y"], t["residual"], post_norm=True, **p)
    s, n = torch.empty_like(t["y"]), torch.empty_like(t["y"])
    missing(ffn.load().ffn_norm, ffn.NormArgs(
        M=M, D=D, groups=1, dtype=ffn.BF16, param_dtype=ffn.F32, kind=ffn.NORM_RMS, flags=3, eps=1e-6, residual_scale=1,
        branch_scale=1, y=t["y"].data_ptr(), residual=t["residual"].data_ptr(), gate=p["gate"].data_ptr(),
        post_weight=p["post_weight"].data_ptr(), pre_weight=p["pre_weight"].data_ptr(), s=s.data_ptr(), n=n.data_ptr()))
    again = ffn.block_norm(t["y"], t["residual"], post_norm=True, **p)
    assert all(torch.equal(a, b) for a, b in zip(want, again))


# warps, a CTA, clusters of two and of eight CTAs, whole groups per part
@pytest.mark.parametrize("M,D,groups", [(300, 64, 1), (300, 1031, 1), (40, 5000, 1), (12, 32640, 1), (600, 520, 300)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_gradient(M, D, groups, kind):
    t, p = norm_inputs(M, D, "bf16", "f32", kind, groups, D)
    p["post_bias"] = p["pre_bias"] = None
    s, _ = ffn.block_norm(t["y"], t["residual"], post_norm=True, kind=kind, **p)
    want = ffn.block_norm_backward(t["ds"], t["dn"], t["y"], s, post_norm=True, kind=kind, **p)
    out = [torch.empty_like(g) for g in want if g is not None]
    a = ffn.NormGradArgs(
        M=M, D=D, groups=groups, dtype=ffn.BF16, param_dtype=ffn.F32, kind=ffn.NORM_KINDS[kind], flags=3, eps=1e-6,
        residual_scale=1, branch_scale=1, ds=t["ds"].data_ptr(), dn=t["dn"].data_ptr(), y=t["y"].data_ptr(),
        s=s.data_ptr(), gate=p["gate"].data_ptr(), post_weight=p["post_weight"].data_ptr(),
        pre_weight=p["pre_weight"].data_ptr(), dresidual=out[0].data_ptr(), dy=out[1].data_ptr(),
        dgate=out[2].data_ptr(), dpost_weight=out[3].data_ptr(), dpre_weight=out[4].data_ptr())
    size = ffn.load().ffn_norm_backward_workspace(ctypes.byref(a))
    workspace = torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)
    a.workspace = workspace.data_ptr()
    missing(ffn.load().ffn_norm_backward, a)
    again = ffn.block_norm_backward(t["ds"], t["dn"], t["y"], s, post_norm=True, kind=kind, **p)
    assert all(x is None and y is None or torch.equal(x, y) for x, y in zip(want, again))
