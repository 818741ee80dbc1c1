"""Rows of calls queued behind other work, with no wait between them: they end, and give
what the same calls give one at a time."""
from __future__ import annotations

import time

import pytest
import torch

from dense_gemm_blackwell_sm_gb300 import ffn, gemm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert ffn.check() == gemm.OK


def ended(limit=20.0):
    """Waits for the stream; a row of calls that does not end ends the run (nothing after it would)."""
    done, began = torch.cuda.Event(), time.monotonic()
    done.record()
    while not done.query():
        if time.monotonic() - began > limit:
            pytest.exit("queued calls did not end in %g s" % limit, returncode=3)
        time.sleep(0.001)


def inputs(M, F, K, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device=DEV) * std).bfloat16()

    return normal(M, K), normal(2 * F, K, std=0.02), normal(M, F), normal(M, 2 * F)


@pytest.mark.parametrize("act", ["gelu_erf", "silu", "gelu_tanh", "relu", "none"])
@pytest.mark.parametrize("M,F,K", [(4096, 14336, 4096), (1024, 4096, 4096), (777, 1097, 1032), (64, 14336, 4096)])
def test_gradients_in_a_row(act, M, F, K):
    x, w, dh, gu = inputs(M, F, K, 1)
    for kept in (gu, None):
        ended()
        want = ffn.gated_backward(dh, x, w, gu=kept, act=act)
        ended()
        # the device is busy making these while the calls are queued
        x2, w2, dh2, gu2 = inputs(M, F, K, 2)
        got = [ffn.gated_backward(dh, x, w, gu=kept, act=act) for _ in range(2)]
        for _ in range(4):
            ffn.gated_backward(dh2, x2, w2, gu=None if kept is None else gu2, act=act)
        got.append(ffn.gated_backward(dh, x, w, gu=kept, act=act))
        ended()
        for g in got:
            assert all(torch.equal(a, b) for a, b in zip(g, want))


@pytest.mark.parametrize("M", [16, 300, 4096])
def test_blocks_in_a_row(M):
    """Norm, projections, their gradients and the norm's gradient, several times over."""
    F, K = 5000, 2048
    x, w, dh, _ = inputs(M, F, K, 3)
    weight = torch.ones(K, device=DEV)

    def block():
        s, n = ffn.block_norm(x, x, pre_weight=weight, post_norm=True)
        h, gu = ffn.gated(n, w, act="gelu_erf", save=True)
        dn, dw = ffn.gated_backward(h, n, w, gu=gu, act="gelu_erf")
        g = ffn.block_norm_backward(None, dn, x, s, pre_weight=weight, post_norm=True)
        return h, dn, dw, g.dresidual, g.dy, g.dpre_weight

    ended()
    want = block()
    ended()
    inputs(M, F, K, 4)
    got = [block() for _ in range(6)]
    ended()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


@pytest.mark.parametrize("M,K,F", [(4096, 4096, 14336), (512, 1024, 4096), (40, 4096, 4096)])
def test_blocks_with_matmul_in_a_row(M, K, F):
    """A stack's forward pass: norm, projections, the library's GEMM, norm, and so on."""
    x, w, _, _ = inputs(M, F, K, 5)
    down = inputs(M, K, F, 6)[1][:K]
    weight = torch.ones(K, device=DEV)

    def stack():
        s, n = ffn.block_norm(x, pre_weight=weight)
        for _ in range(4):
            y = gemm.matmul(ffn.gated(n, w, act="gelu_erf"), down, out_dtype=torch.bfloat16)
            s, n = ffn.block_norm(y, s, post_norm=True, gate=weight, pre_weight=weight)
        return s, n

    ended()
    want = stack()
    ended()
    inputs(M, F, K, 7)
    got = [stack() for _ in range(3)]
    ended()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    assert gemm.gemm_check() == gemm.OK
