"""Pins of the feed-forward block's 64-bit definitions (oracle/ffn.py): closed
forms, PyTorch's own 64-bit operators, and central differences for the gradients."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import ffn as ref

FORMATS = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ["none", "relu", "silu", "gelu_tanh", "gelu_erf"]
TORCH_ACT = {"none": lambda g: g, "relu": torch.relu, "silu": torch.nn.functional.silu,
             "gelu_tanh": lambda g: torch.nn.functional.gelu(g, approximate="tanh"),
             "gelu_erf": torch.nn.functional.gelu}


@pytest.mark.parametrize("name", list(FORMATS))
def test_rounding_is_the_formats(name):
    v = torch.from_numpy(np.exp(_rng(0).uniform(-18, 10, 200000)))
    if name != "f32":
        v = v.float().double()  # torch rounds through fp32
    off = (v.to(FORMATS[name]).double() - v).abs().numpy() / ref.rounding(v.numpy(), name)
    assert 0.999 < off.max() <= 1.0


def _rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("act", ACTS)
def test_activations_are_pytorchs_in_64_bits(act):
    g = torch.linspace(-12, 12, 4001, dtype=torch.float64)
    g = g[g != 0].requires_grad_()
    a = TORCH_ACT[act](g)
    d, = torch.autograd.grad(a.sum(), g)
    va, vd = ref.activation(act, g.detach().numpy())
    assert np.allclose(va, a.detach().numpy(), rtol=0, atol=1e-13)
    assert np.allclose(vd, d.numpy(), rtol=0, atol=1e-13)


@pytest.mark.parametrize("act", ACTS[1:])
def test_largest_slope_and_curvature(act):
    g = np.linspace(-20, 20, 400001)
    _, d = ref.activation(act, g)
    assert np.abs(d).max() <= ref.MAX_SLOPE
    if act != "relu":
        assert np.abs(np.diff(d) / np.diff(g)).max() <= ref.MAX_CURVE


def test_gated_closed_forms():
    r = _rng(1)
    x, w = r.standard_normal((5, 8)), r.standard_normal((14, 8))
    (h, _), (gu, _) = ref.gated(x, w, "none", "bf16")
    assert np.allclose(gu, x @ w.T)
    assert np.allclose(h, (x @ w[:7].T) * (x @ w[7:].T))
    swapped = ref.gated(x, np.concatenate([w[7:], w[:7]]), "silu", "bf16")[0][0]
    assert not np.allclose(swapped, ref.gated(x, w, "silu", "bf16")[0][0])  # gate first, then up


def _numeric(f, v, step=1e-5):
    g = np.zeros_like(v)
    it = np.nditer(v, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        keep = v[i]
        v[i] = keep + step
        hi = f()
        v[i] = keep - step
        lo = f()
        v[i] = keep
        g[i] = (hi - lo) / (2 * step)
    return g


@pytest.mark.parametrize("act", ACTS)
def test_gated_gradient_against_differences(act):
    r = _rng(2)
    x, w, dh = r.standard_normal((3, 8)), r.standard_normal((10, 8)), r.standard_normal((3, 5))
    loss = lambda: float((ref.gated(x, w, act, "f32")[0][0] * dh).sum())  # noqa: E731
    (dx, _), (dw, _) = ref.gated_backward(dh, x, w, None, act, "f32")
    assert np.allclose(dx, _numeric(loss, x), atol=1e-6)
    assert np.allclose(dw, _numeric(loss, w), atol=1e-6)
    kept = ref.gated_backward(dh, x, w, x @ w.T, act, "f32")
    assert np.allclose(kept[0][0], dx) and np.allclose(kept[1][0], dw)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norms_are_pytorchs_in_64_bits(kind):
    r = _rng(3)
    v, w, b = r.standard_normal((6, 17)) * 3 + 1, r.standard_normal(17), r.standard_normal(17)
    got = ref.Unit(v, np.zeros_like(v), kind, 1e-5).affine(w, b)[0]
    t = [torch.from_numpy(a) for a in (v, w, b)]
    want = torch.nn.functional.layer_norm(t[0], (17,), t[1], t[2], 1e-5) if kind == "layer" else \
        torch.nn.functional.rms_norm(t[0], (17,), t[1], 1e-5) + t[2]
    assert np.allclose(got, want.numpy(), atol=1e-13)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("post,pre,groups", [(True, True, 2), (False, True, 1), (True, False, 6), (False, False, 3)])
def test_block_norm_gradient_against_differences(kind, post, pre, groups):
    r = _rng(4)
    M, D = 6, 9
    v = {k: r.standard_normal((M, D)) for k in ("y", "residual", "ds", "dn")}
    p = {k: r.standard_normal(D) + 1 for k in ("post_weight", "post_bias", "pre_weight", "pre_bias")}
    if not post:
        p["post_weight"] = p["post_bias"] = None
    if not pre:
        p["pre_weight"] = p["pre_bias"] = v["dn"] = None
    gate = r.standard_normal((groups, D))
    args = dict(dtype="f32", post=post, gate=gate, pre=pre, kind=kind, eps=1e-3, residual_scale=0.7,
                branch_scale=-1.3, **p)

    def loss():
        s, n = ref.block_norm(v["y"], v["residual"], **args)
        return float((s[0] * v["ds"]).sum() + ((n[0] * v["dn"]).sum() if pre else 0.0))

    s = ref.block_norm(v["y"], v["residual"], **args)[0][0]
    got = ref.block_norm_backward(v["ds"], v["dn"], v["y"], s, **args)
    leaves = [v["residual"], v["y"], gate, p["post_weight"], p["post_bias"], p["pre_weight"], p["pre_bias"]]
    for g, leaf in zip(got, leaves):
        if leaf is None:
            assert g is None
        else:
            assert np.allclose(g[0], _numeric(loss, leaf), atol=2e-6)


def test_planted_mistakes_leave_the_bounds():
    """A dropped term, a swapped half or a wrong mean is far outside the bounds."""
    r = _rng(5)
    x, w = r.standard_normal((9, 64)), r.standard_normal((24, 64)) * 0.2
    h, _ = ref.gated(x, w, "silu", "bf16")
    x2 = x.copy()
    x2[:, 63] = 0
    assert ref.outside(ref.gated(x2, w, "silu", "bf16")[0][0], h)[0] > 50
    assert ref.outside(ref.gated(x, np.roll(w, 12, 0), "silu", "bf16")[0][0], h)[0] > 50
    assert ref.outside(ref.gated(x, w, "gelu_tanh", "bf16")[0][0], h)[0] > 50
    y = r.standard_normal((4, 50)) + 0.1
    args = dict(dtype="bf16", post=True, post_weight=None, post_bias=None, gate=None, pre=True, pre_weight=None,
                pre_bias=None, eps=1e-6)
    s, n = ref.block_norm(y, y[::-1], kind="rms", **args)
    s2, n2 = ref.block_norm(y, y[::-1], kind="layer", **args)
    assert ref.outside(s2[0], s)[0] > 50 and ref.outside(n2[0], n)[0] > 50
    assert ref.outside(s[0], s)[0] == 0
