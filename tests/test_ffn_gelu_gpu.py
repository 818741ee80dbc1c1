"""The erf form of GeLU in its lower tail, where 1 + erf cancels: value and slope against
erfc in 64 bits, relative to their own size.

Gates and up projections are exact (one product each), so only the activation's own
arithmetic and the outputs' rounding are between a result and its definition.  In units
of E = 2^-24: three roundings around the exponent g^2 / 2 (of the square, of the constant
and of their product) move the tail by 1.5 g^2 E relatively; the rest is a few roundings
of one E, the approximate 2^x and 1 / x (4 E and 2 E), and how near the formula comes:
12 E together."""
from __future__ import annotations

import numpy as np
import pytest
import torch
from scipy.special import erfc

from oracle.ffn import rounding
from dense_gemm_blackwell_sm_gb300 import ffn, gemm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T = {"bf16": torch.bfloat16, "f16": torch.float16}
E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert ffn.check() == gemm.OK


def gates(dtype):
    """All gates that the type has in [-9, -0.5], and some above."""
    bits = torch.arange(0, 1 << 15, dtype=torch.int32).to(torch.int16).view(T[dtype]).double()
    low = -bits[(bits >= 0.5) & (bits <= 9.0)]
    low = low[:: max(1, low.numel() // 700)]
    return torch.cat([low, torch.linspace(-0.4, 9, 60).to(T[dtype]).double()])


def operands(M, dtype):
    """x and w with g = the gates and u = 1, each from one product with 1."""
    g = gates(dtype)
    F, K = g.numel(), 8
    x, w = torch.zeros(M, K), torch.zeros(2 * F, K)
    x[:, :2] = 1
    w[:F, 0] = g.float()
    w[F:, 1] = 1
    return g.numpy(), x.to(T[dtype]).to(DEV), w.to(T[dtype]).to(DEV)


def value(g):
    p = 0.5 * erfc(-g / np.sqrt(2.0))
    return g * p, (1.5 * g * g + 12) * E * np.abs(g * p)


def slope(g):
    p, q = 0.5 * erfc(-g / np.sqrt(2.0)), g * np.exp(-0.5 * g * g) / np.sqrt(2 * np.pi)
    return p + q, (1.5 * g * g + 12) * E * p + (1.5 * g * g + 12) * E * np.abs(q) + E * np.abs(p + q)


def within(got, want, bound, dtype, what):
    off = np.abs(got.double().cpu().numpy() - want)
    allowed = bound + rounding(np.abs(want) + bound, dtype)
    assert (off <= allowed).all(), "%s: %d outside, worst %.3g of the bound" % (
        what, int((off > allowed).sum()), float((off / allowed).max()))


@pytest.mark.parametrize("M", [1, 12, 30, 40, 600])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_values(M, dtype):
    g, x, w = operands(M, dtype)
    h, gu = ffn.gated(x, w, act="gelu_erf", save=True)
    assert torch.equal(gu[:, :g.size].double().cpu(), torch.from_numpy(g).expand(M, -1))
    within(h, *value(g), dtype, "h")


@pytest.mark.parametrize("kept", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_slopes(kept, dtype):
    """One token with x = (1, 1, 0, ...) and dh = 1: dw's first column is the slope, its second act(g)."""
    g, x, w = operands(1, dtype)
    gu = ffn.gated(x, w, act="gelu_erf", save=True)[1] if kept else None
    dh = torch.ones(1, g.size, dtype=T[dtype], device=DEV)
    _, dw = ffn.gated_backward(dh, x, w, gu=gu, act="gelu_erf")
    within(dw[:g.size, 0], *slope(g), dtype, "slope")
    within(dw[g.size:, 1], *value(g), dtype, "act")
