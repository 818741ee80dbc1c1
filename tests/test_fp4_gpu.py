"""The product of microscaled 4-bit operands against exact sums in 64 bits: bit for bit where
every partial sum is exact, else within the bounds of an fp32 sum and one rounding."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import ffn as bounds
from oracle import quant as ref
from dense_gemm_blackwell_sm_gb300 import gemm, quant

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
OUT = {"bf16": torch.bfloat16, "f32": torch.float32}
FOUR = ["mxfp4", "nvfp4"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def f64(t):
    return t.double().cpu().numpy()


def codes(rows, cols, fmt, seed, spread=1):
    """A random operand (every code, scales around one) for the oracle."""
    rng = np.random.default_rng(seed)
    w = ref.width(cols)
    c = rng.integers(0, 16, (rows, w)).astype(np.uint8)
    c[:, cols:] = 0
    one = 56 if fmt == "nvfp4" else 127
    step = 8 if fmt == "nvfp4" else 1
    s = one + step * rng.integers(-spread, spread + 1, (rows, w // ref.BLOCK[fmt]))
    row = 2.0 ** rng.integers(-3, 4, rows) if fmt == "nvfp4" else None
    return ref.Operand(c, s.astype(np.uint8), row, fmt, cols)


def device(o):
    row = None if o.row_scale is None else torch.tensor(o.row_scale, dtype=torch.float32, device=DEV)
    return quant.Quantised(torch.tensor(ref.packed(o.codes), device=DEV),
                           torch.tensor(ref.tile(o.scales, o.codes.shape[0]), device=DEV), row, o.format, o.cols)


# one token; tails of every kind; K of less than an MMA, of a whole stage, of more; few tiles and many
SHAPES = [(1, 1, 1), (1, 128, 32), (3, 130, 64), (16, 256, 96), (17, 200, 256), (64, 384, 288), (100, 1000, 512),
          (129, 128, 1024), (130, 520, 4096), (8, 4096, 2048), (700, 3000, 320), (1100, 2500, 608), (300, 6000, 96),
          (65, 9800, 64), (512, 2432, 128), (513, 2432, 128)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("fmt", FOUR)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_exact_sums(shape, fmt, out):
    # scales 1/2, 1 and 2: products are multiples of 2^-4, and with K <= 4096 every partial sum is
    # below 2^24 of those (36 * 4 * 4096 * 16 < 2^24), so the fp32 sum is exact in any order
    M, N, K = shape
    a, b = codes(M, K, fmt, 1), codes(N, K, fmt, 2)
    c = quant.product(device(a), device(b), out_dtype=OUT[out])
    assert quant.check() == gemm.OK
    want = torch.tensor(ref.values(a) @ ref.values(b).T).to(OUT[out]).double().numpy()
    bad = np.argwhere(f64(c) != want)
    assert bad.size == 0, (len(bad), bad[:3], f64(c)[tuple(bad[0])], want[tuple(bad[0])])


@pytest.mark.parametrize("shape", [(1, 4096, 4096), (33, 777, 1056), (513, 2309, 544)])
@pytest.mark.parametrize("fmt", FOUR)
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu_tanh", "gelu_erf"])
def test_quantised_operands_and_epilogue(shape, fmt, act):
    M, N, K = shape
    g = torch.Generator().manual_seed(M + N)
    x = torch.randn(M, K, generator=g).bfloat16()
    w = (torch.randn(N, K, generator=g) * K ** -0.5).bfloat16()
    bias = torch.randn(N, generator=g)
    out = "bf16" if act in ("silu", "none") else "f32"
    res = torch.randn(M, N, generator=g).to(OUT[out])
    wq = quant.quantise(w.to(DEV), fmt)
    kw = dict(out_dtype=OUT[out], bias=bias.to(DEV), act=act, residual=res.to(DEV))
    c = quant.linear(x.to(DEV), wq, **kw)
    assert quant.check() == gemm.OK
    assert torch.equal(c, quant.product(quant.quantise(x.to(DEV), fmt), wq, **kw))
    want = ref.product(ref.quantise(f64(x), fmt), ref.quantise(f64(w), fmt), out, f64(bias), act, f64(res))
    bad, worst = bounds.outside(f64(c), want)
    assert bad == 0, (bad, worst)


@pytest.mark.parametrize("fmt", FOUR)
@pytest.mark.parametrize("M", [5, 300])
def test_scales_belong_to_their_block(fmt, M):
    # one block's scale doubled: only its row or column moves, by that block's share
    N, K = 2600, 512
    a, b = codes(M, K, fmt, 3, 0), codes(N, K, fmt, 4, 0)
    step = 8 if fmt == "nvfp4" else 1
    for o, at in ((a, (M - 1, 5)), (b, (2501, o_cols(fmt, K) - 1)), (b, (70, 2))):
        o.scales[at] += step
    c = f64(quant.product(device(a), device(b), out_dtype=torch.float32))
    assert np.array_equal(c, ref.values(a) @ ref.values(b).T)


def o_cols(fmt, K):
    return K // ref.BLOCK[fmt]


@pytest.mark.parametrize("M,N", [(4, 300), (400, 2700)])
@pytest.mark.parametrize("fmt", FOUR)
def test_strides_out_and_in_place(fmt, M, N):
    K = 160
    a, b = codes(M, K, fmt, 5), codes(N, K, fmt, 6)
    qa, qb = device(a), device(b)
    wide = torch.zeros(M, K // 2 + 48, dtype=torch.uint8, device=DEV)
    wide[:, 16:16 + K // 2] = qa.data
    qa = qa._replace(data=wide[:, 16:16 + K // 2])
    exact = ref.values(a) @ ref.values(b).T
    for dt, pad, off in ((torch.float32, 8, 0), (torch.bfloat16, 3, 1), (torch.bfloat16, 16, 8)):
        room = torch.full((M, N + pad), 7.0, device=DEV, dtype=dt)
        out = room[:, off:off + N]
        got = quant.product(qa, qb, out_dtype=dt, out=out)
        assert got.data_ptr() == out.data_ptr()
        assert np.array_equal(f64(out), f64(torch.tensor(exact).to(dt)))
        assert (room[:, :off] == 7).all() and (room[:, off + N:] == 7).all()
        res = torch.randint(-8, 9, (M, N), generator=torch.Generator().manual_seed(1)).to(dt).to(DEV)
        out.copy_(res)
        quant.product(qa, qb, out_dtype=dt, out=out, residual=out)
        want = torch.tensor(exact + f64(res)).to(dt)
        assert np.array_equal(f64(out), f64(want)) and (room[:, off + N:] == 7).all()


@pytest.mark.parametrize("fmt", FOUR)
@pytest.mark.parametrize("M", [6, 400])
def test_nan_and_infinity_stay_in_their_row(fmt, M):
    N, K = 2600, 96
    g = torch.Generator().manual_seed(7)
    x, w = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g)
    x[2, 50], w[1300, 3] = float("nan"), float("inf")
    c = quant.product(quant.quantise(x.to(DEV), fmt), quant.quantise(w.to(DEV), fmt), out_dtype=torch.float32).cpu()
    hit = torch.zeros(M, N, dtype=torch.bool)
    hit[2], hit[:, 1300] = True, True
    assert torch.equal(torch.isnan(c), hit) and torch.isfinite(c[~hit]).all()


@pytest.mark.parametrize("M", [1, 40, 600])
def test_same_bits_again_streams_and_graph(M):
    N, K = 2560, 1056
    g = torch.Generator().manual_seed(M)
    x, w = torch.randn(M, K, generator=g).bfloat16().to(DEV), torch.randn(N, K, generator=g).bfloat16().to(DEV)
    wq = quant.quantise(w, "nvfp4")
    first = quant.linear(x, wq)
    side = torch.cuda.Stream()
    on_side = quant.linear(x, wq, stream=side, static_b=True)
    side.synchronize()
    assert torch.equal(first, on_side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = quant.linear(x, wq, static_b=True)
        z = quant.linear(y[:, :K].contiguous(), wq, static_b=True)
    for _ in range(3):
        y.zero_()
        z.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, first)
    assert torch.equal(z, quant.linear(first[:, :K].contiguous(), wq))
    assert quant.check() == gemm.OK


@pytest.mark.parametrize("M,N,K", [(0, 40, 64), (3, 0, 64), (5, 70, 0)])
def test_nothing(M, N, K):
    a = quant.quantise(torch.zeros(M, K, dtype=torch.bfloat16, device=DEV), "nvfp4")
    b = quant.quantise(torch.zeros(N, K, dtype=torch.bfloat16, device=DEV), "nvfp4")
    c = quant.product(a, b, bias=torch.ones(N, device=DEV))
    assert c.shape == (M, N) and (c == 1).all()


@pytest.mark.parametrize("M", [4, 700])
def test_a_wait_that_runs_out_is_reported(M):
    a, b = device(codes(M, 512, "nvfp4", 1)), device(codes(3000, 512, "nvfp4", 2))
    quant.product(a, b, timeout_ns=20_000_000, debug_flags=quant.DEBUG_SKIP_ONE_LOAD)
    assert quant.check() == gemm.ERR_DEVICE_TIMEOUT
    assert quant.check() == gemm.OK
    c = quant.product(a, b)
    assert quant.check() == gemm.OK and torch.isfinite(c).all()


def test_refusals_of_tensors():
    a, b = device(codes(4, 64, "nvfp4", 1)), device(codes(6, 64, "nvfp4", 2))
    m = device(codes(6, 64, "mxfp4", 2))
    eight = quant.quantise(torch.zeros(4, 64, device=DEV), "mxe4m3")
    for bad in (lambda: quant.product(a, m), lambda: quant.product(eight, b), lambda: quant.product(a, b._replace(cols=96)),
                lambda: quant.product(a, b._replace(scales=b.scales[:-16])), lambda: quant.product(a, b._replace(scales=None)),
                lambda: quant.product(a, b._replace(row_scale=b.row_scale[:3])),
                lambda: quant.product(a, b._replace(data=b.data[:, :16])),
                lambda: quant.product(a, b, bias=torch.zeros(5, device=DEV)),
                lambda: quant.product(a, b, bias=torch.zeros(6, device=DEV, dtype=torch.bfloat16)),
                lambda: quant.product(a, b, residual=torch.zeros(4, 6, device=DEV)),
                lambda: quant.product(a, b, out_dtype=torch.float16), lambda: quant.product(a, b, act="tanh"),
                lambda: quant.product(a, b, out=torch.zeros(4, 7, device=DEV, dtype=torch.bfloat16)),
                lambda: quant.linear(torch.zeros(4, 32, device=DEV), b),
                lambda: quant.product(a, b._replace(data=b.data.cpu()))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        quant.product(a, b.data)
    # (without row scales they count as one)
    c = quant.product(a._replace(row_scale=None), b, out_dtype=torch.float32)
    assert torch.equal(c, quant.product(a._replace(row_scale=torch.ones(4, device=DEV)), b, out_dtype=torch.float32))


# the tokens' quantisation inside the product (up to 16 of them) and before it: one cluster and
# several CTAs that share a sum, ragged K and N, strided and misaligned tokens
LINEAR = [(1, 1, 1), (1, 130, 33), (5, 128, 96), (16, 300, 520), (16, 4096, 2048), (3, 1000, 4096), (8, 257, 4104),
          (1, 20000, 1000), (17, 130, 96), (4, 9800, 4096),
          (2, 512, 20000)]


@pytest.mark.parametrize("shape", LINEAR)
@pytest.mark.parametrize("fmt", FOUR)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_linear_has_the_bits_of_its_parts(shape, fmt, dtype):
    M, N, K = shape
    gen = torch.Generator().manual_seed(M * 1000 + N + K)
    wide = torch.randn(M, K + 13, generator=gen) * 2.0 ** torch.randint(-6, 7, (M, 1), generator=gen)
    w = quant.quantise(torch.randn(N, K, generator=gen).to(DEV), fmt)
    bias = torch.randn(N, generator=gen).to(DEV)
    residual = torch.randn(M, N, generator=gen).to(DEV)
    for x in (wide[:, :K].contiguous().to(DEV, dtype), wide.to(DEV, dtype)[:, 5:K + 5]):
        q = quant.quantise(x, fmt)
        for kw in (dict(), dict(bias=bias, act="silu", residual=residual, out_dtype=torch.float32, static_b=True)):
            assert torch.equal(quant.linear(x, w, **kw), quant.product(q, w, **kw))


@pytest.mark.parametrize("fmt", FOUR)
def test_linear_with_nan_infinity_and_empty_rows(fmt):
    x = torch.randn(7, 2100, generator=torch.Generator().manual_seed(5)).to(DEV, torch.bfloat16)
    x[1, 3] = float("nan")
    x[2, 2099] = float("inf")
    x[3] = 0
    x[4, 1024:1056] = float("-inf")
    x[5] = -2.0 ** 100
    w = quant.quantise(torch.randn(600, 2100, generator=torch.Generator().manual_seed(6)).to(DEV), fmt)
    got, want = quant.linear(x, w), quant.product(quant.quantise(x, fmt), w)
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())
    assert got[[1, 2, 4]].isnan().all() and not got[[0, 3, 5, 6]].isnan().any() and (got[3] == 0).all()


@pytest.mark.parametrize("fmt", FOUR)
def test_linear_that_waits_too_long_is_reported(fmt):
    w = quant.quantise(torch.randn(512, 1024, device=DEV), fmt)
    x = torch.randn(4, 1024, device=DEV, dtype=torch.bfloat16)
    want = quant.linear(x, w)
    quant.linear(x, w, timeout_ns=20_000_000, debug_flags=quant.DEBUG_SKIP_ONE_LOAD)
    assert quant.check() == gemm.ERR_DEVICE_TIMEOUT
    assert torch.equal(quant.linear(x, w), want) and quant.check() == gemm.OK
