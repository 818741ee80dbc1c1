"""The 4-bit product on CTA pairs (csrc/kernels_fp4_pair.cu): clusters that take several tiles one after
another, with both accumulators, their hand-over and scales of later tiles; every part of the epilogue;
and what surrounds the choice between the kernels (csrc/fp4.h), which each test asks for its shapes."""
from __future__ import annotations

import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import ffn as bounds
from oracle import quant as ref
from dense_gemm_blackwell_sm_gb300 import build as pkg_build
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


RULE = r"""
#include <cstdio>
#include <cstdlib>
#include "fp4.h"

int main(int, char** v) {
  std::printf("%d", dgb::fp4_on_pairs(std::atoll(v[1]), std::atoll(v[2]), std::atoll(v[3]), std::atoi(v[4])));
}
"""


@pytest.fixture(scope="module")
def tiles_a_cluster(tmp_path_factory):
    """How many tiles the cluster with the most of them takes; 0 where the shape is not for pairs."""
    at = tmp_path_factory.mktemp("choice")
    src, exe = at / "rule.cpp", at / "rule"
    src.write_text(RULE)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(pkg_build.nvcc())))
    subprocess.run(["g++", "-std=c++17", "-I", pkg_build.INCLUDE, "-I", pkg_build.CSRC, "-isystem",
                    os.path.join(cuda, "include"), str(src), "-o", str(exe)], check=True)
    sms = torch.cuda.get_device_properties(0).multi_processor_count

    def count(M, N, K):
        run = subprocess.run([str(exe), str(M), str(N), str(ref.width(K)), str(sms)], check=True, capture_output=True, text=True)
        return int(run.stdout) * -(-(-(-M // 256) * -(-N // 256)) // (sms // 2))

    return count


def f64(t):
    return t.double().cpu().numpy()


def codes(rows, cols, fmt, seed, spread=1):
    """A random operand (every code, scales of 1/2, 1 and 2, with spread 0 of 1) for the oracle."""
    rng = np.random.default_rng(seed)
    w = ref.width(cols)
    c = rng.integers(0, 16, (rows, w)).astype(np.uint8)
    c[:, cols:] = 0
    one, step = (56, 8) if fmt == "nvfp4" else (127, 1)
    s = one + step * rng.integers(-spread, spread + 1, (rows, w // ref.BLOCK[fmt]))
    row = 2.0 ** rng.integers(-3, 4, rows) if fmt == "nvfp4" else None
    return ref.Operand(c, s.astype(np.uint8), row, fmt, cols)


def device(o):
    row = None if o.row_scale is None else torch.tensor(o.row_scale, dtype=torch.float32, device=DEV)
    return quant.Quantised(torch.tensor(ref.packed(o.codes), device=DEV),
                           torch.tensor(ref.tile(o.scales, o.codes.shape[0]), device=DEV), row, o.format, o.cols)


def times(a, b):
    """a b^T in 64 bits, on the device.  (Products are multiples of 2^-4 and below 2^8 times the rows'
    scales, all sums of up to 4096 of them exact.)"""
    return torch.tensor(ref.values(a), device=DEV) @ torch.tensor(ref.values(b), device=DEV).T


# three to five tiles a cluster of 76: a last column of tiles that holds 8 columns (its common columns
# lie past N, so that a warp hands back and goes on at once), whole tiles, ragged ones; one stage of K,
# more stages than fit
SEVERAL = [(16384, 1032, 64), (4352, 4200, 96), (16500, 1001, 1312), (5000, 4096, 288)]


@pytest.mark.parametrize("shape", SEVERAL)
@pytest.mark.parametrize("fmt", FOUR)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_several_tiles_of_a_cluster(shape, fmt, out, tiles_a_cluster):
    M, N, K = shape
    assert tiles_a_cluster(*shape) >= 3
    a, b = codes(M, K, fmt, 1), codes(N, K, fmt, 2)
    qa, qb, want = device(a), device(b), times(a, b).to(OUT[out])
    for _ in range(3):
        c = quant.product(qa, qb, out_dtype=OUT[out])
        assert quant.check() == gemm.OK
        assert torch.equal(c, want), torch.nonzero(c != want)[:3]


@pytest.mark.parametrize("fmt", FOUR)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("K", [96, 2080])
def test_a_wait_that_runs_out_ends_every_role(fmt, out, K, tiles_a_cluster):
    # each CTA's first copy is left out: what waits for it gives up, then what waits for that, over
    # several tiles; the calls behind it are whole
    M, N = 4352, 4200
    assert tiles_a_cluster(M, N, K) >= 3
    a, b = codes(M, K, fmt, 3), codes(N, K, fmt, 4)
    qa, qb, want = device(a), device(b), times(a, b).to(OUT[out])
    quant.product(qa, qb, out_dtype=OUT[out], timeout_ns=20_000_000, debug_flags=quant.DEBUG_SKIP_ONE_LOAD)
    c = quant.product(qa, qb, out_dtype=OUT[out])
    assert quant.check() == gemm.ERR_DEVICE_TIMEOUT
    assert torch.equal(c, want) and quant.check() == gemm.OK
    assert torch.equal(quant.product(qa, qb, out_dtype=OUT[out]), want) and quant.check() == gemm.OK


# rows of C that start on 16-byte boundaries (stored and read by whole pieces) and rows that do not; one
# tile a cluster with every activation, several with both outputs
EPILOGUES = [(shape, act, out) for shape in ((1100, 2504, 1056), (1100, 2500, 1056))
             for act, out in (("none", "bf16"), ("relu", "f32"), ("silu", "bf16"), ("gelu_tanh", "f32"), ("gelu_erf", "bf16"))]
EPILOGUES += [(shape, act, out) for shape in ((4352, 4200, 544), (4352, 4203, 544)) for act, out in (("relu", "f32"), ("silu", "bf16"))]


@pytest.mark.parametrize("shape,act,out", EPILOGUES)
@pytest.mark.parametrize("fmt", FOUR)
def test_epilogue(shape, fmt, act, out, tiles_a_cluster):
    M, N, K = shape
    assert tiles_a_cluster(*shape) == (1 if M == 1100 else 4)
    g = torch.Generator().manual_seed(M + N)
    x = torch.randn(M, K, generator=g).bfloat16()
    w = (torch.randn(N, K, generator=g) * K ** -0.5).bfloat16()
    bias, res = torch.randn(N, generator=g), torch.randn(M, N, generator=g).to(OUT[out])
    wq = quant.quantise(w.to(DEV), fmt)
    kw = dict(out_dtype=OUT[out], bias=bias.to(DEV), act=act, residual=res.to(DEV))
    c = quant.linear(x.to(DEV), wq, **kw)
    assert quant.check() == gemm.OK
    assert torch.equal(c, quant.product(quant.quantise(x.to(DEV), fmt), wq, **kw))
    want = ref.product(ref.quantise(f64(x), fmt), ref.quantise(f64(w), fmt), out, f64(bias), act, f64(res))
    bad, worst = bounds.outside(f64(c), want)
    assert bad == 0, (bad, worst)


@pytest.mark.parametrize("M,N", [(1100, 2500), (4352, 4200)])
@pytest.mark.parametrize("fmt", FOUR)
def test_strides_out_and_in_place(fmt, M, N, tiles_a_cluster):
    K = 160
    assert tiles_a_cluster(M, N, K) >= 1
    a, b = codes(M, K, fmt, 5), codes(N, K, fmt, 6)
    qa, qb, exact = device(a), device(b), times(a, b)
    wide = torch.zeros(M, K // 2 + 48, dtype=torch.uint8, device=DEV)
    wide[:, 16:16 + K // 2] = qa.data
    qa = qa._replace(data=wide[:, 16:16 + K // 2])
    tall = torch.zeros(N, K // 2 + 16, dtype=torch.uint8, device=DEV)
    tall[:, :K // 2] = qb.data
    qb = qb._replace(data=tall[:, :K // 2])
    for dt, pad, off in ((torch.float32, 8, 0), (torch.float32, 5, 2), (torch.bfloat16, 3, 1), (torch.bfloat16, 20, 8)):
        room = torch.full((M, N + pad), 7.0, device=DEV, dtype=dt)
        out = room[:, off:off + N]
        got = quant.product(qa, qb, out_dtype=dt, out=out)
        assert got.data_ptr() == out.data_ptr()
        assert torch.equal(out, exact.to(dt))
        assert (room[:, :off] == 7).all() and (room[:, off + N:] == 7).all()
        res = torch.randint(-8, 9, (M, N), generator=torch.Generator().manual_seed(1)).to(dt).to(DEV)
        out.copy_(res)
        quant.product(qa, qb, out_dtype=dt, out=out, residual=out)
        assert torch.equal(out, (exact + res.double()).to(dt)) and (room[:, off + N:] == 7).all()
        assert quant.check() == gemm.OK


@pytest.mark.parametrize("fmt", FOUR)
@pytest.mark.parametrize("M,N", [(1100, 2600), (4352, 4200)])
def test_nan_and_infinity_stay_in_their_row(fmt, M, N, tiles_a_cluster):
    K = 96
    assert tiles_a_cluster(M, N, K) >= 1
    g = torch.Generator().manual_seed(7)
    x, w = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g)
    x[M - 2, 50], w[1300, 3] = float("nan"), float("inf")
    c = quant.product(quant.quantise(x.to(DEV), fmt), quant.quantise(w.to(DEV), fmt), out_dtype=torch.float32).cpu()
    hit = torch.zeros(M, N, dtype=torch.bool)
    hit[M - 2], hit[:, 1300] = True, True
    assert torch.equal(torch.isnan(c), hit) and torch.isfinite(c[~hit]).all()


@pytest.mark.parametrize("fmt", FOUR)
def test_scales_belong_to_their_block(fmt, tiles_a_cluster):
    M, N, K = 4352, 4200, 512
    assert tiles_a_cluster(M, N, K) >= 3
    a, b = codes(M, K, fmt, 3, 0), codes(N, K, fmt, 4, 0)
    last, step = K // ref.BLOCK[fmt] - 1, 8 if fmt == "nvfp4" else 1
    for o, at in ((a, (M - 1, 5)), (a, (2177, last)), (b, (N - 1, last)), (b, (70, 2))):
        o.scales[at] += step
    assert torch.equal(quant.product(device(a), device(b), out_dtype=torch.float32), times(a, b).float())


@pytest.mark.parametrize("fmt", FOUR)
def test_same_bits_again_streams_and_graph(fmt, tiles_a_cluster):
    M, N, K = 4352, 4200, 1056
    assert tiles_a_cluster(M, N, K) >= 3
    g = torch.Generator().manual_seed(M)
    x, w = torch.randn(M, K, generator=g).bfloat16().to(DEV), torch.randn(N, K, generator=g).bfloat16().to(DEV)
    wq, res = quant.quantise(w, fmt), torch.randn(M, N, generator=g).bfloat16().to(DEV)
    first = quant.linear(x, wq, residual=res)
    side = torch.cuda.Stream()
    on_side = quant.linear(x, wq, residual=res, stream=side, static_b=True)
    side.synchronize()
    assert torch.equal(first, on_side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = quant.linear(x, wq, residual=res, static_b=True)
        z = quant.linear(y[:, :K].contiguous(), wq, residual=y, static_b=True)
    want = quant.linear(first[:, :K].contiguous(), wq, residual=first)
    for _ in range(3):
        y.zero_()
        z.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, first) and torch.equal(z, want)
    assert quant.check() == gemm.OK


# 65 to 256 tokens with long sums: single CTAs and clusters of them, scales of one, so that sums of up to
# 14336 products (multiples of 1/4, 36 at most) are exact
@pytest.mark.parametrize("shape", [(65, 300, 4128), (100, 1200, 5024), (130, 1000, 14336), (200, 520, 8192), (256, 4096, 14336)])
@pytest.mark.parametrize("fmt", FOUR)
def test_long_sums_of_some_tokens(shape, fmt, tiles_a_cluster):
    M, N, K = shape
    assert tiles_a_cluster(*shape) == 0
    a, b = codes(M, K, fmt, 1, 0), codes(N, K, fmt, 2, 0)
    for out in OUT.values():
        assert torch.equal(quant.product(device(a), device(b), out_dtype=out), times(a, b).to(out))
    x = torch.randn(M, K - 7, generator=torch.Generator().manual_seed(K)).bfloat16().to(DEV)
    w = quant.quantise(torch.randn(N, K - 7, generator=torch.Generator().manual_seed(N)).to(DEV), fmt)
    assert torch.equal(quant.linear(x, w), quant.product(quant.quantise(x, fmt), w))
    assert quant.check() == gemm.OK


def plain(rows, fmt, seed, cols=32):
    """An operand of `rows` rows of one block, or two, with scales of one, made on the device."""
    data = torch.randint(0, 256, (rows, cols // 2), generator=torch.Generator(DEV).manual_seed(seed), dtype=torch.uint8, device=DEV)
    scales = torch.full((quant.scale_bytes(rows, cols, fmt),), 56 if fmt == "nvfp4" else 127, dtype=torch.uint8, device=DEV)
    return quant.Quantised(data, scales, None, fmt, cols)


def tail(q, rows):
    """Its last rows, from a scale block's first one."""
    assert (q.data.shape[0] - rows) % 128 == 0
    return q._replace(data=q.data[-rows:], scales=q.scales[-quant.scale_bytes(rows, q.cols, q.format):])


# outputs past 2^31 elements, at every kernel: the last rows and columns as they are alone (the sums are exact)
@pytest.mark.parametrize("M,N", [(66048, 32896), (66048, 32801), (64, (1 << 25) + 256), (16, (1 << 27) + 128)])
@pytest.mark.parametrize("fmt", FOUR)
def test_outputs_past_two_to_the_31_elements(M, N, fmt, tiles_a_cluster):
    assert M * N > 2 ** 31 and (tiles_a_cluster(M, N, 32) > 100) == (M > 64)
    a, b = plain(M, fmt, 1), plain(N, fmt, 2)
    c = quant.product(a, b)
    assert quant.check() == gemm.OK
    rows, cols = min(M, 256), 256 if N % 128 == 0 else 256 + N % 128
    want = quant.product(tail(a, rows), tail(b, cols))
    assert torch.equal(c[-rows:, -cols:], want) and torch.equal(c[:128, -cols:], quant.product(a, tail(b, cols))[:128])
    assert torch.equal(c[-rows:, :256], quant.product(tail(a, rows), b)[:, :256])
    # a linear layer whose tokens are its own values: small whole numbers keep their codes
    del c, want
    x = torch.randint(-3, 4, (M, 32), generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    x[:, :] = torch.where(x.abs() == 3, x * 2, x)
    c, alone = quant.linear(x, b), quant.linear(x[-rows:], tail(b, cols))
    assert quant.check() == gemm.OK and torch.equal(c[-rows:, -cols:], alone)


@pytest.mark.parametrize("M,N", [(1100, 2500), (1100, 2501), (4352, 4203), (4352, 4254)])
@pytest.mark.parametrize("fmt", FOUR)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_what_lies_beside_the_output_stays(M, N, fmt, out, tiles_a_cluster):
    # columns that end inside a 16-byte piece of a wider array whose rows are aligned
    K, dt = 96, OUT[out]
    assert tiles_a_cluster(M, N, K) >= 1
    a, b = codes(M, K, fmt, 5), codes(N, K, fmt, 6)
    qa, qb, exact = device(a), device(b), times(a, b)
    room = torch.full((M + 1, (N + 40) // 16 * 16), 7.0, device=DEV, dtype=dt)
    place = room[:M, 16:16 + N]
    res = torch.randint(-8, 9, (M, N), generator=torch.Generator().manual_seed(1)).to(dt).to(DEV)
    for residual in (None, res, place):
        before = 0 if residual is None else residual.double()
        quant.product(qa, qb, out_dtype=dt, out=place, residual=residual)
        assert quant.check() == gemm.OK
        assert torch.equal(place, (exact + before).to(dt))
        assert (room[:, :16] == 7).all() and (room[:, 16 + N:] == 7).all() and (room[M] == 7).all()
