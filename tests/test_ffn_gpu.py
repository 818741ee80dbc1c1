"""GPU parity of the feed-forward block's operators against their 64-bit
definitions, element by element within the derived bounds of oracle/ffn.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import ffn as ref
from dense_gemm_blackwell_sm_gb300 import ffn, gemm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ["none", "relu", "silu", "gelu_tanh", "gelu_erf"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert ffn.check() == gemm.OK


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def randn(gen, *shape, dtype, std=1.0, mean=0.0, pitch=None):
    """Random rows; with `pitch` (elements) as a view of a wider array filled with NaN."""
    v = (torch.randn(shape, generator=gen) * std + mean).to(T[dtype]).to(DEV)
    if pitch is None:
        return v
    wide = torch.full((shape[0], pitch), float("nan"), dtype=T[dtype], device=DEV)
    wide[:, :shape[1]] = v
    return wide[:, :shape[1]]


def assert_within(got, want, what):
    bad, worst = ref.outside(f64(got), want)
    assert bad == 0, "%s: %d elements outside, worst %.3g of the bound" % (what, bad, worst)


# ------------------------------------------------------------ gated projections

# one token, decode batches, the edges of 16 / 32 / 128 / 256 / 512-row tiles, widths and depths
# around tiles of 64 and 128, odd F, a K of one 16-byte chunk and one past a stage
GATED = [(1, 256, 128), (1, 1, 8), (2, 77, 1000), (3, 128, 64), (5, 33, 2056), (8, 300, 512), (9, 64, 72),
         (15, 129, 264), (16, 1000, 640), (17, 96, 136), (20, 100, 72),
         (24, 513, 264), (25, 9, 8), (29, 1541, 2056), (32, 300, 4104), (33, 257, 520), (64, 1543, 200), (127, 128, 64),
         (128, 256, 1032), (129, 130, 192), (255, 511, 328), (256, 127, 64), (257, 640, 72), (300, 1541, 520),
         (511, 88, 136), (513, 260, 256), (1100, 1031, 392)]


def gated_inputs(M, F, K, dtype, seed, **pitches):
    gen = torch.Generator().manual_seed(seed)
    x = randn(gen, M, K, dtype=dtype, pitch=pitches.get("x"))
    w = randn(gen, 2 * F, K, dtype=dtype, std=1.3 / K ** 0.5, pitch=pitches.get("w"))
    return gen, x, w


@pytest.mark.parametrize("M,F,K", GATED)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gated(M, F, K, dtype):
    act = ACTS[(M + F) % 5]
    _, x, w = gated_inputs(M, F, K, dtype, M + F)
    want_h, want_gu = ref.gated(f64(x), f64(w), act, dtype)
    h, gu = ffn.gated(x, w, act=act, save=True)
    assert_within(h, want_h, "h")
    assert_within(gu, want_gu, "gu")
    alone = ffn.gated(x, w, act=act)
    assert torch.equal(alone, h)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [4, 28, 150, 520])
def test_gated_activations(act, M):
    """Each activation in each kernel, gates from deep saturation to zero."""
    F, K = 200, 64
    gen, x, w = gated_inputs(M, F, K, "f16", 7)
    w[:F] *= torch.logspace(-3, 1.6, F, device=DEV, dtype=torch.float32)[:, None].half()
    assert_within(ffn.gated(x, w, act=act), ref.gated(f64(x), f64(w), act, "f16")[0], act)
    dh = randn(gen, M, F, dtype="f16")
    for got, want in zip(ffn.gated_backward(dh, x, w, act=act),
                         ref.gated_backward(f64(dh), f64(x), f64(w), None, act, "f16")):
        assert_within(got, want, act)


@pytest.mark.parametrize("M", [1, 7, 13, 22, 32, 40, 300, 700])
def test_integers_are_exact(M):
    """Small integers: every fp32 sum and product is exact, so the outputs must be too."""
    F, K = 130, 256
    gen = torch.Generator().manual_seed(M)
    x = torch.randint(-2, 3, (M, K), generator=gen).bfloat16().to(DEV)
    w = torch.randint(-1, 2, (2 * F, K), generator=gen).bfloat16().to(DEV)
    h, gu = ffn.gated(x, w, act="relu", save=True)
    exact = x.double().cpu() @ w.double().cpu().t()
    assert torch.equal(gu.cpu(), exact.bfloat16())
    assert torch.equal(h.cpu(), (exact[:, :F].clamp(min=0) * exact[:, F:]).bfloat16())
    gu = torch.randint(-3, 4, (M, 2 * F), generator=gen).bfloat16().to(DEV)
    dh = torch.randint(-2, 3, (M, F), generator=gen).bfloat16().to(DEV)
    dx, dw = ffn.gated_backward(dh, x, w, gu=gu, act="relu")
    g, u, d = gu[:, :F].double().cpu(), gu[:, F:].double().cpu(), dh.double().cpu()
    dgu = torch.cat([d * u * (g > 0), d * g.clamp(min=0)], 1)
    assert torch.equal(dx.cpu(), (dgu @ w.double().cpu()).bfloat16())
    assert torch.equal(dw.cpu(), (dgu.t() @ x.double().cpu()).bfloat16())


GRADS = [(1, 40, 64), (2, 33, 200), (17, 128, 136), (64, 257, 72), (130, 96, 520), (255, 301, 256), (300, 512, 264),
         (514, 129, 1000), (777, 1097, 1032), (1030, 200, 128)]


@pytest.mark.parametrize("M,F,K", GRADS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kept", [True, False])
def test_gated_backward(M, F, K, dtype, kept):
    act = ACTS[(M + F + kept) % 5]
    gen, x, w = gated_inputs(M, F, K, dtype, M * 3 + F)
    dh = randn(gen, M, F, dtype=dtype)
    gu = ffn.gated(x, w, act=act, save=True)[1] if kept else None
    want = ref.gated_backward(f64(dh), f64(x), f64(w), f64(gu), act, dtype)
    dx, dw = ffn.gated_backward(dh, x, w, gu=gu, act=act)
    assert_within(dx, want[0], "dx")
    assert_within(dw, want[1], "dw")
    only_x, none = ffn.gated_backward(dh, x, w, gu=gu, act=act, need_dw=False)
    assert none is None and torch.equal(only_x, dx)
    none, only_w = ffn.gated_backward(dh, x, w, gu=gu, act=act, need_dx=False)
    assert none is None and torch.equal(only_w, dw)


@pytest.mark.parametrize("M,F,K", [(1, 2000, 64), (20, 5003, 264), (100, 7001, 520), (130, 14336, 128), (300, 1541, 520),
                                   (777, 1097, 1032), (513, 3000, 72)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gated_backward_long_reductions(M, F, K, dtype):
    """dx of few tokens through wide layers: slices of its reduction, joined."""
    gen, x, w = gated_inputs(M, F, K, dtype, F)
    dh, gu = randn(gen, M, F, dtype=dtype), randn(gen, M, 2 * F, dtype=dtype)
    dx, dw = ffn.gated_backward(dh, x, w, gu=gu)
    want = ref.gated_backward(f64(dh), f64(x), f64(w), f64(gu), "silu", dtype)
    assert_within(dx, want[0], "dx")
    assert_within(dw, want[1], "dw")
    assert torch.equal(dx, ffn.gated_backward(dh, x, w, gu=gu, need_dw=False)[0])
    assert torch.equal(dw, ffn.gated_backward(dh, x, w, gu=gu, need_dx=False)[1])


def test_gated_gradient_against_differences():
    """The kernel's gradient along a direction is the 64-bit loss's central difference."""
    M, F, K, act = 70, 90, 128, "silu"
    gen, x, w = gated_inputs(M, F, K, "f16", 11)
    dh = randn(gen, M, F, dtype="f16")
    dx, dw = ffn.gated_backward(dh, x, w, act=act)
    X, W, D = f64(x), f64(w), f64(dh)
    rng = np.random.default_rng(0)
    vx, vw = rng.standard_normal(X.shape), rng.standard_normal(W.shape) * 0.1

    def loss(t):
        return (ref.gated(X + t * vx, W + t * vw, act, "f16")[0][0] * D).sum()

    step = 1e-4
    want = (loss(step) - loss(-step)) / (2 * step)
    (rx, bx), (rw, bw) = ref.gated_backward(D, X, W, None, act, "f16")
    got = (f64(dx) * vx).sum() + (f64(dw) * vw).sum()
    assert abs(got - want) <= (bx * np.abs(vx)).sum() + (bw * np.abs(vw)).sum() + 1e-6 * abs(want)
    # the bound above is a worst case; the errors are independent, so far less of it is used
    assert abs(got - want) <= 8 * (np.sqrt(((bx * vx) ** 2).sum()) + np.sqrt(((bw * vw) ** 2).sum()))


@pytest.mark.parametrize("M", [3, 12, 31, 100, 600])
def test_gated_pitched_rows(M):
    """Rows wider than their use (and odd pitches of h, gu and dh), with NaN in between:
    nothing outside the arrays is read into a result or written."""
    F, K, dtype = 133, 200, "bf16"
    gen, x, w = gated_inputs(M, F, K, dtype, M, x=216, w=256)
    dh = randn(gen, M, F, dtype=dtype, pitch=135)
    wide_h = torch.full((M, 141), 7.0, dtype=T[dtype], device=DEV)
    wide_gu = torch.full((M, 2 * F + 3), 7.0, dtype=T[dtype], device=DEV)
    h, gu = ffn.gated(x, w, act="silu", save=True, out=wide_h[:, :F], gu=wide_gu[:, :2 * F])
    want_h, want_gu = ref.gated(f64(x), f64(w), "silu", dtype)
    assert_within(h, want_h, "h")
    assert_within(gu, want_gu, "gu")
    assert bool((wide_h[:, F:] == 7).all()) and bool((wide_gu[:, 2 * F:] == 7).all())
    want = ref.gated_backward(f64(dh), f64(x), f64(w), f64(gu), "silu", dtype)
    for got, b in zip(ffn.gated_backward(dh, x, w, gu=gu, act="silu"), want):
        assert_within(got, b, "gradient")


@pytest.mark.parametrize("M", [1, 6, 20, 30, 300])
def test_unaligned_output(M):
    """An output that starts 2 bytes off a 16-byte boundary."""
    F, K = 128, 128
    _, x, w = gated_inputs(M, F, K, "f16", M)
    flat = torch.full((M * F + 2,), 7.0, dtype=torch.float16, device=DEV)
    h = ffn.gated(x, w, out=flat[1:-1].view(M, F))
    assert torch.equal(h, ffn.gated(x, w))
    assert flat[0] == 7 and flat[-1] == 7


@pytest.mark.parametrize("M", [2, 18, 40, 700])
def test_values_that_are_not_finite_stay_in_their_row_and_column(M):
    F, K = 150, 136
    gen, x, w = gated_inputs(M, F, K, "bf16", 5)
    clean = ffn.gated(x, w, act="silu")
    x2, w2 = x.clone(), w.clone()
    x2[1, 3] = float("nan")
    w2[F + 7, 0] = float("inf")
    h = ffn.gated(x2, w2, act="silu")
    assert bool(h[1].isnan().all())
    rest = torch.ones(M, F, dtype=torch.bool, device=DEV)
    rest[1], rest[:, 7] = False, False
    assert torch.equal(h[rest], clean[rest])
    assert not bool(h[:, 7].isfinite().any())


@pytest.mark.parametrize("M", [5, 12, 27, 90, 530])
def test_gated_is_reproducible(M):
    F, K = 260, 328
    gen, x, w = gated_inputs(M, F, K, "bf16", 9)
    dh = randn(gen, M, F, dtype="bf16")
    first = [*ffn.gated(x, w, save=True), *ffn.gated_backward(dh, x, w)]
    for _ in range(3):
        again = [*ffn.gated(x, w, save=True), *ffn.gated_backward(dh, x, w)]
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_gated_without_tokens():
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), torch.ones(20, 64, dtype=torch.bfloat16, device=DEV)
    h, gu = ffn.gated(x, w, save=True)
    assert h.shape == (0, 10) and gu.shape == (0, 20)
    dx, dw = ffn.gated_backward(h, x, w, gu=gu)
    assert dx.shape == (0, 64) and dw.shape == (20, 64) and bool((dw == 0).all())


def test_gated_on_another_stream_and_in_a_graph():
    M, F, K = 200, 300, 256
    gen, x, w = gated_inputs(M, F, K, "bf16", 3)
    dh = randn(gen, M, F, dtype="bf16")
    want = [*ffn.gated(x, w, save=True), *ffn.gated_backward(dh, x, w)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [*ffn.gated(x, w, save=True, stream=side), *ffn.gated_backward(dh, x, w, stream=side)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [*ffn.gated(x, w, save=True), *ffn.gated_backward(dh, x, w)]
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_gated_chain_on_one_stream():
    """Calls that read what the call before wrote, back to back."""
    M, K = 96, 256
    gen = torch.Generator().manual_seed(4)
    w = randn(gen, 2 * K, K, dtype="bf16", std=1.6 / K ** 0.5)
    small, large = randn(gen, 4, K, dtype="bf16"), randn(gen, M, K, dtype="bf16")
    for x in (small, large):
        want = x
        for _ in range(6):
            want = ffn.gated(want, w, act="gelu_tanh")
            torch.cuda.synchronize()
        got = x
        for _ in range(6):
            got = ffn.gated(got, w, act="gelu_tanh")
        assert torch.equal(got, want)


def test_large_offsets():
    """Outputs and pre-activations past 2^31 elements."""
    M, F, K = 70000, 15400, 64
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(M, K, generator=gen, device=DEV).bfloat16()
    w = (torch.randn(2 * F, K, generator=gen, device=DEV) * 0.2).bfloat16()
    h, gu = ffn.gated(x, w, act="silu", save=True)
    assert gu.numel() > 2 ** 31
    for rows in (slice(0, 3), slice(M // 2, M // 2 + 3), slice(M - 3, M)):
        want_h, want_gu = ref.gated(f64(x[rows]), f64(w), "silu", "bf16")
        assert_within(h[rows], want_h, "h")
        assert_within(gu[rows], want_gu, "gu")
    dh = h
    dx, dw = ffn.gated_backward(dh, x, w, gu=gu, act="silu")
    rows = slice(M - 3, M)
    want = ref.gated_backward(f64(dh[rows]), f64(x[rows]), f64(w), f64(gu[rows]), "silu", "bf16")
    assert_within(dx[rows], want[0], "dx")
    del h, gu, dh, dx, dw


@pytest.mark.parametrize("M,F,K", [(33, 1, 8), (40, 3, 64), (130, 17, 72), (256, 16, 8), (600, 5, 136)])
def test_gated_narrow(M, F, K):
    """Fewer features than a tile's columns, and reductions of one block, in the tiled kernel."""
    gen, x, w = gated_inputs(M, F, K, "f16", F)
    want_h, want_gu = ref.gated(f64(x), f64(w), "silu", "f16")
    h, gu = ffn.gated(x, w, save=True)
    assert_within(h, want_h, "h")
    assert_within(gu, want_gu, "gu")
    dh = randn(gen, M, F, dtype="f16")
    for kept in (gu, None):
        want = ref.gated_backward(f64(dh), f64(x), f64(w), f64(kept), "silu", "f16")
        for got, b in zip(ffn.gated_backward(dh, x, w, gu=kept), want):
            assert_within(got, b, "gradient")


@pytest.mark.parametrize("M,F,K", [(100, 300, 512), (300, 4000, 128), (2000, 4000, 256)])
def test_a_copy_that_never_comes_ends_in_a_status(M, F, K):
    """One operand copy left out: the bounded waits run out, the call's kernels return,
    ffn.check reports it once, and the next call is whole."""
    gen, x, w = gated_inputs(M, F, K, "bf16", 1)
    dh = randn(gen, M, F, dtype="bf16")
    want = ffn.gated(x, w)
    grads = ffn.gated_backward(dh, x, w)
    assert ffn.check() == gemm.OK
    ffn.gated(x, w, timeout_ns=50_000_000, debug_flags=ffn.DEBUG_SKIP_ONE_LOAD)
    assert ffn.check() == gemm.ERR_DEVICE_TIMEOUT
    assert ffn.check() == gemm.OK
    ffn.gated_backward(dh, x, w, timeout_ns=50_000_000, debug_flags=ffn.DEBUG_SKIP_ONE_LOAD)
    assert ffn.check() == gemm.ERR_DEVICE_TIMEOUT
    assert torch.equal(ffn.gated(x, w), want)
    assert all(torch.equal(a, b) for a, b in zip(ffn.gated_backward(dh, x, w), grads))
    assert ffn.check() == gemm.OK


def test_gated_refusals_on_the_gpu():
    _, x, w = gated_inputs(4, 16, 64, "bf16", 0)
    with pytest.raises(ValueError):
        ffn.gated(x, w, act="swish")
    with pytest.raises(gemm.GemmError) as e:
        ffn.gated(x, w, act=9)
    assert e.value.status == gemm.ERR_INVALID_ARG
    with pytest.raises(gemm.GemmError) as e:
        ffn.gated(x[:, :60], w[:, :60])
    assert e.value.status == gemm.ERR_UNSUPPORTED_SHAPE
    flat = torch.zeros(4 * 64 + 8, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(gemm.GemmError) as e:
        ffn.gated(flat[4:-4].view(4, 64), w)
    assert e.value.status == gemm.ERR_MISALIGNED
    with pytest.raises(ValueError):
        ffn.gated(x, w, out=torch.zeros(4, 15, dtype=torch.bfloat16, device=DEV))


@pytest.mark.parametrize("M", [1, 8, 9, 16, 17, 25])
@pytest.mark.parametrize("F,K", [(2440, 264), (1208, 72), (2424, 8), (1217, 4096)])
def test_few_tokens_over_the_device(M, F, K):
    """As many CTAs as SMs, twice as many and a few more; K of fewer pieces than warps."""
    gen, x, w = gated_inputs(M, F, K, "bf16", F)
    want_h, want_gu = ref.gated(f64(x), f64(w), "gelu_erf", "bf16")
    h, gu = ffn.gated(x, w, act="gelu_erf", save=True)
    assert_within(h, want_h, "h")
    assert_within(gu, want_gu, "gu")


def test_calls_keep_nothing():
    """Outputs, temporaries and refused calls leave no memory and no references behind."""
    import sys
    _, x, w = gated_inputs(40, 24, 64, "bf16", 3)
    gate = torch.ones(64, device=DEV)
    dh = torch.ones(40, 24, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()

    def calls():
        h, gu = ffn.gated(x, w, save=True)
        ffn.gated_backward(dh, x, w, gu=gu)
        ffn.gated(x, w, out=h, gu=gu, stream=side)
        s, n = ffn.block_norm(x, gate=gate, post_norm=True, pre_weight=gate)
        ffn.block_norm_backward(n, s, x, s, gate=gate, post_norm=True, pre_weight=gate, stream=side.cuda_stream)
        for bad in (lambda: ffn.gated(x, w[:7]), lambda: ffn.gated(x, w, act=9), lambda: ffn.block_norm(x, x[:2]),
                    lambda: ffn.block_norm(x, gate=gate[:3])):
            with pytest.raises((ValueError, gemm.GemmError)):
                bad()
        torch.cuda.synchronize()
        return h, gu

    h, gu = calls()
    assert ffn.gated(x, w, out=h) is h
    held = torch.cuda.memory_allocated()
    counts = [sys.getrefcount(t) for t in (x, w, gate, dh, h, None)][:-1]
    for _ in range(20):
        calls()
    assert torch.cuda.memory_allocated() <= held  # (what another stream used is freed some calls later)
    assert [sys.getrefcount(t) for t in (x, w, gate, dh, h, None)][:-1] == counts


# ------------------------------------------------------------------------ norms

# rows of one element, around warps and 8-element accesses, powers of two, odd lengths, the longest
NORMS = [(1, 1), (3, 2), (5, 7), (4, 8), (2, 31), (7, 64), (1, 255), (9, 256), (6, 1000), (5, 1001), (3, 1024),
         (130, 513), (4, 2048), (8, 4096), (1, 4096), (2, 5000), (3, 8192), (2, 8193), (1, 12288), (2, 16384),
         (1, 20001), (2, 32768)]


def norm_inputs(M, D, dtype, param, kind, groups, seed, affine=True):
    gen = torch.Generator().manual_seed(seed)
    vec = lambda mean: randn(gen, D, dtype=param, std=0.3, mean=mean) if affine else None  # noqa: E731
    bias = kind == "layer"
    t = dict(y=randn(gen, M, D, dtype=dtype, std=1.5, mean=0.3), residual=randn(gen, M, D, dtype=dtype, std=3.0),
             ds=randn(gen, M, D, dtype=dtype), dn=randn(gen, M, D, dtype=dtype))
    p = dict(post_weight=vec(1.0), post_bias=vec(0.0) if bias else None, pre_weight=vec(1.0),
             pre_bias=vec(0.0) if bias else None,
             gate=randn(gen, groups, D, dtype=param, std=0.4, mean=0.6) if groups else None)
    return t, p


def ref_norm(t, p, dtype, **kw):
    return ref.block_norm(f64(t["y"]), f64(t["residual"]), dtype, **{k: f64(v) for k, v in p.items()}, **kw)


def ref_norm_grad(t, p, s, dtype, **kw):
    return ref.block_norm_backward(f64(t["ds"]), f64(t["dn"]), f64(t["y"]), f64(s), dtype,
                                   **{k: f64(v) for k, v in p.items()}, **kw)


def check_norm(t, p, dtype, kind, post=True, pre=True, eps=1e-6, **scales):
    kw = dict(kind=kind, eps=eps, **scales)
    s, n = ffn.block_norm(t["y"], t["residual"], post_norm=post, pre_norm=pre, **p, **kw)
    want_s, want_n = ref_norm(t, p, dtype, post=post, pre=pre, **kw)
    assert_within(s, want_s, "s")
    if pre:
        assert_within(n, want_n, "n")
    else:
        assert n is None
    got = ffn.block_norm_backward(t["ds"], t["dn"], t["y"], s, post_norm=post, pre_norm=pre, **p, **kw)
    want = ref_norm_grad(t, p, s, dtype, post=post, pre=pre, **kw)
    for name, g, b in zip(got._fields, got, want):
        assert (g is None) == (b is None), name
        if g is not None:
            assert_within(g, b, name)
    return s, n, got


@pytest.mark.parametrize("M,D", NORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_block_norm(M, D, dtype, kind):
    param = "f32" if (M + D) % 2 else dtype
    groups = 1 if M % 2 else M // 2
    t, p = norm_inputs(M, D, dtype, param, kind, groups, M + D)
    check_norm(t, p, dtype, kind)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("groups", [0, 1, 4, 12])
def test_block_norm_parts(post, pre, affine, groups):
    """Every combination of parts, with scales, on vector and scalar widths."""
    for D in (264, 131):
        t, p = norm_inputs(12, D, "bf16", "bf16", "layer", groups, D, affine)
        if not post:
            p["post_weight"] = p["post_bias"] = None
        if not pre:
            p["pre_weight"] = p["pre_bias"] = t["dn"] = None
        if groups == 4:
            t["residual"] = None
        if groups == 1 and pre:
            t["ds"] = None
        check_norm(t, p, "bf16", "layer", post=post, pre=pre, residual_scale=0.5, branch_scale=-1.5)


@pytest.mark.parametrize("M,groups", [(1, 1), (40, 40), (600, 1), (600, 3), (600, 100), (1000, 8), (2500, 5),
                                      (5000, 2500)])
@pytest.mark.parametrize("D", [96, 520])
def test_sums_over_rows(M, groups, D):
    """Parameter gradients over many rows, gates whose rows end anywhere in a CTA's share."""
    t, p = norm_inputs(M, D, "f16", "f32", "layer", groups, M)
    _, _, first = check_norm(t, p, "f16", "layer")
    s, _ = ffn.block_norm(t["y"], t["residual"], post_norm=True, kind="layer", **p)
    for _ in range(2):
        again = ffn.block_norm_backward(t["ds"], t["dn"], t["y"], s, post_norm=True, kind="layer", **p)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("M,D", [(5000, 33), (4000, 255), (2000, 1031), (1300, 2032), (1301, 2039), (1300, 2047),
                                 (1300, 2048), (1300, 2049), (900, 4095), (900, 4096), (901, 4097), (700, 5001),
                                 (500, 9003)])
@pytest.mark.parametrize("dtype,kind", [("bf16", "rms"), ("f16", "layer"), ("f32", "rms")])
def test_many_rows(M, D, dtype, kind):
    """More rows than a device holds at once, around the widths where a row's split changes."""
    t, p = norm_inputs(M, D, dtype, "f32", kind, 1, M + D)
    check_norm(t, p, dtype, kind)


def test_norm_large_offsets():
    """Rows past 2^31 elements: the last rows' values, and sums over rows that are zero but there."""
    M, D = 131080, 16392
    gen = torch.Generator(device=DEV).manual_seed(3)
    t = {k: torch.zeros((M, D), dtype=torch.bfloat16, device=DEV) for k in ("y", "residual", "ds", "dn")}
    assert t["y"].numel() > 2 ** 31
    last = slice(M - 3, M)
    for v in t.values():
        v[last] = torch.randn((3, D), generator=gen, device=DEV).bfloat16()
    p = dict(post_weight=torch.randn(D, generator=gen, device=DEV), post_bias=None, pre_bias=None,
             pre_weight=torch.randn(D, generator=gen, device=DEV), gate=torch.randn(D, generator=gen, device=DEV))
    s, n = ffn.block_norm(t["y"], t["residual"], post_norm=True, **p)
    got = ffn.block_norm_backward(t["ds"], t["dn"], t["y"], s, post_norm=True, **p)
    few = {k: v[last] for k, v in t.items()}
    one = {**p, "gate": p["gate"][None]}
    kw = dict(post=True, pre=True, kind="rms", eps=1e-6)
    want_s, want_n = ref_norm(few, one, "bf16", **kw)
    want = ref_norm_grad(few, one, s[last], "bf16", **kw)
    assert_within(s[last], want_s, "s")
    assert_within(n[last], want_n, "n")
    for name, g, b in zip(got._fields, got, want):
        if g is not None:
            assert_within(g[last] if g.shape == (M, D) else g.reshape(b[0].shape), b, name)
    assert not s[:M - 3].any() and not n[:M - 3].any() and not got.dy[:M - 3].any()


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_rows_of_zeros_and_constants(kind):
    """A padding row of zeros and a constant row: eps alone is under the root."""
    t, p = norm_inputs(4, 200, "f32", "f32", kind, 1, 2)
    t["y"][0] = 0
    t["residual"][0] = 0
    p["post_bias"] = None
    t["y"][1] = 2.5
    check_norm(t, p, "f32", kind, eps=1e-3)


def test_large_mean_keeps_its_deviation():
    """Values far from zero with a small spread: the variance is taken around the mean."""
    t, p = norm_inputs(5, 1024, "f32", "f32", "layer", 1, 8)
    t["y"] = t["y"] * 0.01 + 300
    s, n, _ = check_norm(t, p, "f32", "layer")
    want = torch.nn.functional.layer_norm(t["y"].double(), (1024,), p["post_weight"].double(), p["post_bias"].double(),
                                          1e-6) * p["gate"].double() + t["residual"].double()
    assert float((s - want).abs().max()) < 0.05


@pytest.mark.parametrize("D", [256, 333, 9000])
def test_norm_in_place_and_pitched(D):
    t, p = norm_inputs(9, D, "bf16", "f32", "rms", 3, D)
    kw = dict(post_norm=True, kind="rms", **p)
    s, n = ffn.block_norm(t["y"], t["residual"], **kw)
    y2, r2 = t["y"].clone(), t["residual"].clone()
    s2, n2 = ffn.block_norm(y2, r2, s=r2, n=y2, **kw)
    assert s2 is r2 and n2 is y2 and torch.equal(s, r2) and torch.equal(n, y2)
    wide = {k: torch.full((9, D + pad), float("nan"), dtype=torch.bfloat16, device=DEV)
            for k, pad in (("y", 8), ("residual", 3), ("ds", 1), ("dn", 24))}
    for k, v in wide.items():
        v[:, :D] = t[k]
    out_s, out_n = (torch.full((9, D + pad), 7.0, dtype=torch.bfloat16, device=DEV) for pad in (8, 5))
    ffn.block_norm(wide["y"][:, :D], wide["residual"][:, :D], s=out_s[:, :D], n=out_n[:, :D], **kw)
    assert torch.equal(out_s[:, :D], s) and torch.equal(out_n[:, :D], n)
    assert bool((out_s[:, D:] == 7).all()) and bool((out_n[:, D:] == 7).all())
    want = ffn.block_norm_backward(t["ds"], t["dn"], t["y"], s, **kw)
    got = ffn.block_norm_backward(wide["ds"][:, :D], wide["dn"][:, :D], wide["y"][:, :D], out_s[:, :D], **kw)
    assert all(torch.equal(a, b) for a, b in zip(want, got) if a is not None)


def test_norm_unaligned_rows():
    """Rows that start one element past a 16-byte boundary."""
    t, p = norm_inputs(6, 512, "f16", "f32", "layer", 2, 1)
    flat = {k: torch.zeros(6 * 512 + 1, dtype=torch.float16, device=DEV) for k in t}
    for k, v in flat.items():
        v[1:] = t[k].reshape(-1)
    shifted = {k: v[1:].view(6, 512) for k, v in flat.items()}
    s, n, g = check_norm(shifted, p, "f16", "layer")
    s2, n2, g2 = check_norm(t, p, "f16", "layer")
    assert torch.equal(s, s2) and torch.equal(n, n2)
    p["pre_weight"] = torch.cat([p["pre_weight"][:1], p["pre_weight"]])[1:]
    check_norm(t, p, "f16", "layer")


def test_norm_without_rows_and_without_needs():
    e = torch.empty(0, 32, dtype=torch.float16, device=DEV)
    w = torch.ones(32, device=DEV)
    s, n = ffn.block_norm(e, e, pre_weight=w)
    assert s.shape == n.shape == (0, 32)
    g = ffn.block_norm_backward(e, e, e, s, pre_weight=w, gate=w)
    assert g.dresidual.shape == (0, 32) and bool((g.dpre_weight == 0).all()) and bool((g.dgate == 0).all())
    t, p = norm_inputs(5, 64, "f16", "f32", "rms", 1, 1)
    s, n = ffn.block_norm(t["y"], t["residual"], need_s=False, post_norm=True, **p)
    assert s is None and n is not None
    s, _ = ffn.block_norm(t["y"], t["residual"], post_norm=True, **p)
    full = ffn.block_norm_backward(t["ds"], t["dn"], t["y"], s, post_norm=True, **p)
    some = ffn.block_norm_backward(t["ds"], t["dn"], t["y"], s, post_norm=True, need_dparams=False,
                                   need_dresidual=False, **p)
    assert some.dresidual is None and some.dgate is None and torch.equal(some.dy, full.dy)


def test_norm_values_that_are_not_finite_stay_in_their_row():
    t, p = norm_inputs(5, 300, "bf16", "f32", "layer", 1, 1)
    s, n = ffn.block_norm(t["y"], t["residual"], post_norm=True, kind="layer", **p)
    t["y"][2, 17] = float("inf")
    t["residual"][3, 5] = float("nan")
    s2, n2 = ffn.block_norm(t["y"], t["residual"], post_norm=True, kind="layer", **p)
    keep = torch.tensor([0, 1, 4], device=DEV)
    assert torch.equal(s2[keep], s[keep]) and torch.equal(n2[keep], n[keep])
    assert bool(n2[2].isnan().all()) and bool(n2[3].isnan().all())


def test_norm_on_another_stream_and_in_a_graph():
    t, p = norm_inputs(300, 640, "bf16", "f32", "rms", 3, 6)
    run = lambda **kw: [*ffn.block_norm(t["y"], t["residual"], post_norm=True, **p, **kw)]  # noqa: E731
    want = run()
    back = lambda s, **kw: [g for g in ffn.block_norm_backward(t["ds"], t["dn"], t["y"], s, post_norm=True,  # noqa
                                                                **p, **kw) if g is not None]
    want += back(want[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = run(stream=side)
    got += back(got[0], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
        got += back(got[0])
    for g in got:
        g.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_norm_gradient_against_differences():
    t, p = norm_inputs(12, 100, "f32", "f32", "layer", 3, 5)
    s, _, got = check_norm(t, p, "f32", "layer")
    rng = np.random.default_rng(1)
    leaves = {"y": f64(t["y"]), "residual": f64(t["residual"]), **{k: f64(v) for k, v in p.items()}}
    along = {k: rng.standard_normal(v.shape) for k, v in leaves.items()}

    def loss(h):
        v = {k: leaves[k] + h * along[k] for k in leaves}
        a, b = ref.block_norm(v.pop("y"), v.pop("residual"), "f32", post=True, pre=True, kind="layer", eps=1e-6, **v)
        return (a[0] * f64(t["ds"])).sum() + (b[0] * f64(t["dn"])).sum()

    want = (loss(1e-5) - loss(-1e-5)) / 2e-5
    pairs = zip(("residual", "y", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias"), got)
    total = sum((f64(g) * along[k]).sum() for k, g in pairs)
    assert abs(total - want) <= 1e-4 * abs(want) + 1e-3


def test_norm_refusals_on_the_gpu():
    t, p = norm_inputs(4, 64, "bf16", "f32", "rms", 1, 1)
    with pytest.raises(gemm.GemmError) as e:
        ffn.block_norm(t["y"], t["residual"], kind=7)
    assert e.value.status == gemm.ERR_INVALID_ARG
    wide = torch.zeros(1, 32769, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(gemm.GemmError) as e:
        ffn.block_norm(wide, wide)
    assert e.value.status == gemm.ERR_UNSUPPORTED_SHAPE
    with pytest.raises(ValueError):
        ffn.block_norm(t["y"], t["residual"], s=torch.zeros(4, 64, device=DEV))
    with pytest.raises(ValueError):
        ffn.block_norm(t["y"].int(), t["residual"].int())
