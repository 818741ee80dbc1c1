"""The low-precision operators as they are used together: a feed-forward stack run with 8- and
4-bit products, a layer's training step, and the whole captured in a graph."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import ffn as bounds
from oracle import quant as ref
from dense_gemm_blackwell_sm_gb300 import ffn, gemm, quant

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FOUR = ["mxfp4", "nvfp4"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def f64(t):
    return t.double().cpu().numpy()


def normal(*shape, seed, std=1.0, to=torch.bfloat16):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(to).to(DEV)


def kept(q):
    """A Quantised of the device as the oracle's Operand."""
    rows, cols = q.data.shape[0], q.cols
    b = q.data.view(torch.uint8).cpu().numpy()
    codes = np.stack([b & 15, b >> 4], 2).reshape(rows, -1) if q.format in FOUR else b
    scales = None
    if q.scales is not None:
        n = codes.shape[1] // ref.BLOCK[q.format]
        r, c = np.meshgrid(np.arange(rows), np.arange(n), indexing="ij")
        at = ((r // 128) * (-(-n // 4)) + c // 4) * 512 + (r % 32) * 16 + ((r // 32) % 4) * 4 + c % 4
        scales = q.scales.cpu().numpy()[at]
    return ref.Operand(codes, scales, None if q.row_scale is None else f64(q.row_scale), q.format, cols)


@pytest.mark.parametrize("M", [1, 200])
@pytest.mark.parametrize("fmt", FOUR)
def test_norm_into_product(fmt, M):
    # norm with a quantised output -> 4-bit product with activation -> product added to the stream
    D, F = 520, 1000
    y, s = normal(M, D, seed=1), normal(M, D, seed=2)
    w1, w2 = normal(F, D, seed=3, std=D ** -0.5), normal(D, F, seed=4, std=F ** -0.5)
    q1, q2 = quant.quantise(w1, fmt), quant.quantise(w2, fmt)
    s, n = quant.norm_quantise(y, s, format=fmt)
    h = quant.product(n, q1, act="silu", static_b=True)
    out = quant.linear(h, q2, residual=s, static_b=True)
    assert quant.check() == gemm.OK
    # each step from what the one before gave
    want = ref.product(kept(n), ref.quantise(f64(w1), fmt), "bf16", act="silu")
    assert bounds.outside(f64(h), want)[0] == 0
    want = ref.product(ref.quantise(f64(h), fmt), ref.quantise(f64(w2), fmt), "bf16", residual=f64(s))
    assert bounds.outside(f64(out), want)[0] == 0


@pytest.mark.parametrize("fmt", ["e4m3", "mxe4m3"])
def test_eight_bit_operands_into_gemm(fmt):
    # what the quantiser and the norm write is what the library's own 8-bit products read
    M, N, D = 300, 520, 416
    x, w = normal(M, D, seed=1), normal(N, D, seed=2, std=D ** -0.5)
    _, a = quant.norm_quantise(x, format=fmt)
    b = quant.quantise(w, fmt)
    c = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    plan = gemm.Plan(M, N, D, gemm.dtype_code(fmt, "bf16"))
    if fmt == "e4m3":
        plan.run_epilogue(a.data, b.data, c, scale_a=a.row_scale, scale_b=b.row_scale)
    else:
        plan.run_mx(a.data, b.data, c, a.scales, b.scales)
    assert plan.check() == gemm.OK
    want = ref.product(kept(a), kept(b), "bf16")
    assert bounds.outside(f64(c), want)[0] == 0


@pytest.mark.parametrize("shape", [(1, 64, 96), (40, 300, 200), (515, 1097, 264), (300, 2600, 1032), (0, 40, 64)])
@pytest.mark.parametrize("fmt", FOUR)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_linear_backward_is_its_formula(shape, fmt, dtype):
    M, N, K = shape
    dy, x = normal(M, N, seed=1, std=0.1, to=dtype), normal(M, K, seed=2, to=dtype)
    w = normal(N, K, seed=3, std=K ** -0.5, to=dtype)
    out = torch.float32 if dtype == torch.float32 else torch.bfloat16
    name = "f32" if out == torch.float32 else "bf16"
    dx, dw = quant.linear_backward(dy, x, w, format=fmt, out_dtype=out)
    assert quant.check() == gemm.OK
    q = lambda v: ref.quantise(v, fmt)  # noqa: E731
    for got, want in ((dx, ref.product(q(f64(dy)), q(f64(w).T), name)), (dw, ref.product(q(f64(dy).T), q(f64(x).T), name))):
        bad, worst = bounds.outside(f64(got), want)
        assert bad == 0, (bad, worst)
    only, none = quant.linear_backward(dy, None, w, format=fmt, need_dw=False, out_dtype=out)
    assert none is None and torch.equal(only, dx)
    none, only = quant.linear_backward(dy, x, None, format=fmt, need_dx=False, out_dtype=out)
    assert none is None and torch.equal(only, dw)


@pytest.mark.parametrize("fmt", FOUR)
def test_linear_backward_against_differences(fmt):
    # L = sum(dy * (x w^T)) is linear in x and in w, so differences are exact; the gradients may be
    # off by what quantisation moves the operands: |dx - dy w| <= |dy - Q dy| |w| + |Q dy| |w - Q w|
    M, N, K = 70, 96, 130
    dy, x, w = normal(M, N, seed=1), normal(M, K, seed=2), normal(N, K, seed=3)
    dx, dw = (f64(t) for t in quant.linear_backward(dy, x, w, format=fmt, out_dtype=torch.float32))
    loss = lambda x, w: (f64(dy) * (x @ w.T)).sum()  # noqa: E731
    q = lambda v: ref.values(ref.quantise(v, fmt))[:, :v.shape[1]]  # noqa: E731
    rng = np.random.default_rng(0)
    for got, left, right, which in ((dx, f64(dy), f64(w).T, 0), (dw, f64(dy).T, f64(x).T, 1)):
        room = np.abs(left - q(left)) @ np.abs(right).T + np.abs(q(left)) @ np.abs(right - q(right)).T
        for _ in range(4):
            d = rng.normal(size=got.shape)
            at = [f64(x), f64(w)]
            moved = list(at)
            moved[which] = at[which] + d
            difference = loss(*moved) - loss(*at)
            assert abs((got * d).sum() - difference) <= (room * np.abs(d)).sum() * (1 + 1e-6) + 1e-3


def test_gradient_of_the_norm():
    # the norm's gradient is block_norm's; here against differences of s and n in 64 bits
    M, D = 6, 64
    y, res, w = normal(M, D, seed=1, to=torch.float32), normal(M, D, seed=2, to=torch.float32), normal(D, seed=3, to=torch.float32)
    ds, dn = normal(M, D, seed=4, to=torch.float32), normal(M, D, seed=5, to=torch.float32)
    s, _ = quant.norm_quantise(y, res, w, format="nvfp4")
    g = ffn.block_norm_backward(ds, dn, y, s, pre_weight=w)

    def loss(y, res, w):
        (s, _), (n, _) = ref.norm(y, res, w, "f32", 1e-6)
        return (f64(ds) * s).sum() + (f64(dn) * n).sum()

    at = [f64(y), f64(res), f64(w)]
    rng = np.random.default_rng(1)
    for which, grad in ((0, g.dy), (1, g.dresidual), (2, g.dpre_weight)):
        d = rng.normal(size=at[which].shape)
        up, down = list(at), list(at)
        up[which], down[which] = at[which] + 1e-5 * d, at[which] - 1e-5 * d
        want = (loss(*up) - loss(*down)) / 2e-5
        assert abs((f64(grad) * d).sum() - want) <= 1e-4 * np.abs(f64(grad) * d).sum() + 1e-4


@pytest.mark.parametrize("M", [2, 384])
def test_a_block_in_a_graph(M):
    D, F = 512, 1536
    w1, w2 = quant.quantise(normal(F, D, seed=1, std=D ** -0.5), "nvfp4"), quant.quantise(normal(D, F, seed=2, std=F ** -0.5), "nvfp4")
    y, s = normal(M, D, seed=3), normal(M, D, seed=4)

    def block(y, s):
        s, n = quant.norm_quantise(y, s, format="nvfp4")
        h = quant.product(n, w1, act="gelu_tanh", static_b=True)
        y = quant.linear(h, w2, static_b=True)
        s, n = quant.norm_quantise(y, s, format="nvfp4")
        return s, quant.linear(quant.product(n, w1, act="gelu_tanh", static_b=True), w2, static_b=True)

    want = block(y, s)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block(y, s)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(y, s)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # two at once, each on its own stream
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        second = [block(y, s) for _ in range(5)]
    first = [block(y, s) for _ in range(5)]
    torch.cuda.synchronize()
    for pair in first + second:
        assert all(torch.equal(a, b) for a, b in zip(pair, want))
    assert quant.check() == gemm.OK


@pytest.mark.parametrize("D", [1001, 97, 33])
@pytest.mark.parametrize("fmt", ["e4m3", "mxe4m3"])
def test_ragged_eight_bit_operands_into_gemm(fmt, D):
    # rows are kept with their padding: the plan's K is their width
    M, N, K = 130, 264, quant.width(D)
    assert K == -(-D // 32) * 32
    x, w = normal(M, D, seed=1), normal(N, D, seed=2, std=D ** -0.5)
    a, b = quant.quantise(x, fmt), quant.quantise(w, fmt)
    assert a.data.shape == (M, K) and a.cols == D
    c = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    plan = gemm.Plan(M, N, K, gemm.dtype_code(fmt, "bf16"))
    if fmt == "e4m3":
        plan.run_epilogue(a.data, b.data, c, scale_a=a.row_scale, scale_b=b.row_scale)
    else:
        plan.run_mx(a.data, b.data, c, a.scales, b.scales)
    assert plan.check() == gemm.OK
    bad, worst = bounds.outside(f64(c), ref.product(ref.quantise(f64(x), fmt), ref.quantise(f64(w), fmt), "bf16"))
    assert bad == 0, (bad, worst)
