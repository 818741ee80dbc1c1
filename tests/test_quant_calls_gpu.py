"""Calls of the low-precision operands that belong together: several arrays at once, operands that
share memory with others, tiles' edges, host threads, replays of two graphs in turn."""
from __future__ import annotations

import ctypes
import threading

import pytest
import torch

from dense_gemm_blackwell_sm_gb300 import ffn, gemm, quant

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FOUR = ["mxfp4", "nvfp4"]
CODE = {torch.float16: ffn.F16, torch.bfloat16: ffn.BF16, torch.float32: ffn.F32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def normal(*shape, seed, to=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(to).to(DEV)


def same(a, b):
    parts = [(a.data, b.data), (a.scales, b.scales), (a.row_scale, b.row_scale)]
    return all((x is None and y is None) or torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in parts)


def rows_call(x, fmt, transpose):
    """The arguments of a call, and what it will have written."""
    lib = quant.load()
    rows, cols = (x.shape[1], x.shape[0]) if transpose else x.shape
    code = quant.FORMATS[fmt]
    data = torch.full((rows, lib.quant_row_bytes(cols, code)), 0xa5, dtype=torch.uint8, device=DEV)
    scales = None if fmt == "e4m3" else torch.full((lib.quant_scale_bytes(rows, cols, code),), 0xa5, dtype=torch.uint8, device=DEV)
    row_scale = torch.full((rows,), 7.0, device=DEV) if fmt in ("e4m3", "nvfp4") else None
    a = quant.RowsArgs(rows=x.shape[0], cols=x.shape[1], dtype=CODE[x.dtype], format=code, transpose=int(transpose),
                       x=x.data_ptr(), data=data.data_ptr(), scales=scales.data_ptr() if scales is not None else None,
                       row_scale=row_scale.data_ptr() if row_scale is not None else None, ld_x=x.stride(0))
    work = torch.empty(max(16, lib.quant_rows_workspace(ctypes.byref(a))), dtype=torch.uint8, device=DEV)
    a.workspace = work.data_ptr()
    return a, quant.Quantised(data, scales, row_scale, fmt, cols), work


SIX = [(300, 520), (1, 1), (64, 2000), (1000, 33), (257, 129), (96, 640)]


@pytest.mark.parametrize("fmt", list(quant.FORMATS))
@pytest.mark.parametrize("mixed", [False, True])
def test_many_arrays_are_as_one_by_one(fmt, mixed):
    # six arrays by columns (more than go in a launch); mixed: types and directions change in between
    other = "nvfp4" if fmt == "mxfp4" else "mxfp4"
    calls = []
    for i, shape in enumerate(SIX):
        dtype = [torch.bfloat16, torch.float16, torch.float32][i % 3] if mixed else torch.bfloat16
        f = other if mixed and i == 3 else fmt
        calls.append((normal(*shape, seed=i, to=dtype), f, not (mixed and i % 2)))
    made = [rows_call(*c) for c in calls]
    args = (quant.RowsArgs * len(made))(*[m[0] for m in made])
    stream = gemm._stream_ptr(None)
    assert quant.load().quant_rows_many(args, len(made), stream) == gemm.OK
    assert quant.check() == gemm.OK
    for (x, f, t), (_, got, _) in zip(calls, made):
        want = quant.quantise(x, f, transpose=t)
        assert same(got, quant.Quantised(want.data.view(torch.uint8), *want[1:])), (x.shape, f, t)
    # nothing of a list with a refused call in it is launched
    for m in made:
        m[1].data.fill_(0x5a)
    args[5].format = 9
    assert quant.load().quant_rows_many(args, len(made), stream) == gemm.ERR_UNSUPPORTED_DTYPE
    torch.cuda.synchronize()
    assert all((m[1].data == 0x5a).all() for m in made)


@pytest.mark.parametrize("M", [63, 64, 65, 127, 128, 129, 192])
@pytest.mark.parametrize("fmt", FOUR)
def test_rows_do_not_depend_on_their_tile(fmt, M):
    # 64 tokens a tile, half of a block of scales, and tiles of 256: a row's product is its own
    x, w = normal(M, 352, seed=M), normal(300, 352, seed=2)
    a, b = quant.quantise(x, fmt), quant.quantise(w, fmt)
    c = quant.product(a, b, out_dtype=torch.float32)
    # Two orders of one sum of K products: each is off by K 2^-23 of the sum of their magnitudes at
    # most (adds that may truncate), and a quantised magnitude is at most twice its value's.
    bound = 2 * 352 * 2.0 ** -23 * 4 * (x.float().abs() @ w.float().abs().T)
    for rows in ([0], [M - 1], [M // 2, M - 1]):
        want = quant.product(quant.quantise(x[rows], fmt), b, out_dtype=torch.float32)
        assert ((c[rows] - want).abs() <= bound[rows]).all()


@pytest.mark.parametrize("fmt", FOUR)
@pytest.mark.parametrize("M", [3, 40])
def test_linear_between_columns_of_one_array(fmt, M):
    buf = normal(M, 1024, seed=1)
    x, out = buf[:, :256], buf[:, 256:256 + 264]
    w = quant.quantise(normal(264, 256, seed=2), fmt)
    want, keep = quant.linear(x.clone(), w), buf.clone()
    quant.linear(x, w, out=out)
    assert torch.equal(out, want)
    assert torch.equal(buf[:, :256], keep[:, :256]) and torch.equal(buf[:, 520:], keep[:, 520:])
    w = quant.quantise(normal(256, 256, seed=3), fmt)
    for bad in (x, buf[:, 128:384]):
        with pytest.raises(gemm.GemmError):
            quant.linear(x, w, out=bad)


@pytest.mark.parametrize("fmt", FOUR)
def test_two_graphs_in_turn(fmt):
    # each has its own workspace; replays in turn, and on two streams, keep both results
    w = [quant.quantise(normal(640, 520, seed=i), fmt) for i in range(2)]
    x = [normal(M, 520, seed=9 + M) for M in (2, 300)]
    want = [quant.linear(a, b, act="silu") for a, b in zip(x, w)]
    wide = [quant.quantise(a, fmt, transpose=True) for a in x]
    graphs, got = [], []
    for a, b in zip(x, w):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append((quant.linear(a, b, act="silu", static_b=True), quant.quantise(a, fmt, transpose=True)))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert quant.check() == gemm.OK
    for (y, q), t, u in zip(got, want, wide):
        assert torch.equal(y, t) and same(q, u)


def test_two_host_threads():
    x, w = normal(200, 1000, seed=1), normal(700, 1000, seed=2)
    q = quant.quantise(w, "nvfp4")
    want = quant.linear(x, q)
    results, failed = [], []

    def work():
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                y = [quant.linear(x, q, static_b=True) for _ in range(50)]
            s.synchronize()
            results.append(y)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and all(torch.equal(y, want) for r in results for y in r) and len(results) == 2


@pytest.mark.parametrize("fmt", list(quant.FORMATS))
def test_odd_pitches_of_the_norm(fmt):
    # rows of y, of the residual and of s on different boundaries; s in place of the residual
    M, D = 70, 1001
    y = normal(M, D + 4, seed=1)[:, 1:D + 1]
    r = normal(M, D + 7, seed=2)[:, 2:D + 2]
    weight = normal(D, seed=3, to=torch.float32)
    s0, q0 = quant.norm_quantise(y.contiguous(), r.contiguous(), weight, format=fmt)
    s1, q1 = quant.norm_quantise(y, r, weight, format=fmt)
    assert torch.equal(s0, s1) and same(q0, q1)
    s2, q2 = quant.norm_quantise(y, r, weight, format=fmt, s=r)
    assert s2.data_ptr() == r.data_ptr() and torch.equal(r, s0) and same(q0, q2)
    none, q3 = quant.norm_quantise(y, s0, None, format=fmt, need_s=False)
    assert none is None and q3.data.shape == q0.data.shape


@pytest.mark.parametrize("fmt", FOUR)
@pytest.mark.parametrize("M,N,K", [(3, 40, 0), (40, 40, 0), (0, 40, 64), (3, 0, 64), (0, 0, 0)])
def test_linear_of_nothing(fmt, M, N, K):
    x, w = torch.zeros(M, K, device=DEV), quant.quantise(torch.zeros(N, K, device=DEV), fmt)
    bias, residual = normal(N, seed=1, to=torch.float32), normal(M, N, seed=2, to=torch.float32)
    y = quant.linear(x, w, bias=bias, residual=residual, out_dtype=torch.float32)
    assert torch.equal(y, (bias + residual) if M and N else residual)
    assert quant.check() == gemm.OK


@pytest.mark.parametrize("fmt", FOUR)
def test_linear_of_one_token_and_the_largest_and_smallest_values(fmt):
    # magnitudes at the ends of the types: the kernel that quantises tokens itself, as rows
    w = quant.quantise(normal(256, 512, seed=1), fmt)
    for dtype, values in ((torch.float16, (65504.0, 6e-8)), (torch.bfloat16, (2.0 ** 100, 2.0 ** -120)), (torch.float32, (2.0 ** 100, 2.0 ** -120))):
        for v in values:
            x = torch.zeros(1, 512, device=DEV, dtype=dtype)
            x[0, 7], x[0, 8], x[0, 300] = v, -v, v
            assert torch.equal(quant.linear(x, w, out_dtype=torch.float32),
                               quant.product(quant.quantise(x, fmt), w, out_dtype=torch.float32))


@pytest.mark.parametrize("fmt", list(quant.FORMATS))
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_no_values_with_a_pitch(fmt, transpose, dtype):
    # (what lies behind the address is NaN, none of it the array's)
    x = torch.full((100, 64), float("nan"), dtype=dtype, device=DEV)
    empty = x[:, :0]
    a, got, _ = rows_call(empty, fmt, transpose)
    a.ld_x = 64
    assert a.rows == 100 and a.cols == 0
    assert quant.load().quant_rows(ctypes.byref(a), gemm._stream_ptr(None)) == gemm.OK
    assert quant.check() == gemm.OK
    want = quant.quantise(torch.empty(100, 0, dtype=dtype, device=DEV), fmt, transpose=transpose)
    assert same(got, quant.Quantised(want.data.view(torch.uint8), *want[1:]))
    assert not got.data.any() and (transpose or got.data.shape[0] == 100)


@pytest.mark.parametrize("fmt", FOUR)
@pytest.mark.parametrize("M", [3, 40])
def test_linear_of_no_values_with_a_pitch(fmt, M):
    # (in one kernel and in two)
    N, lib = 130, quant.load()
    x = torch.full((M, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    w = quant.quantise(torch.empty(N, 0, device=DEV), fmt)
    bias, c = normal(N, seed=1, to=torch.float32), torch.full((M, N), 7.0, device=DEV)
    a = quant.LinearArgs(M=M, N=N, K=0, dtype=ffn.BF16, format=quant.FORMATS[fmt], out_dtype=ffn.F32, x=x.data_ptr(),
                         b=w.data.data_ptr(), scales_b=w.scales.data_ptr(),
                         row_scale_b=w.row_scale.data_ptr() if w.row_scale is not None else None, bias=bias.data_ptr(),
                         c=c.data_ptr(), ld_x=64)
    work = torch.empty(max(256, lib.quant_linear_workspace(ctypes.byref(a))), dtype=torch.uint8, device=DEV)
    a.workspace = work.data_ptr()
    assert lib.quant_linear(ctypes.byref(a), gemm._stream_ptr(None)) == gemm.OK
    assert quant.check() == gemm.OK
    assert torch.equal(c, bias.expand(M, N))


@pytest.mark.parametrize("fmt", FOUR)
def test_the_time_of_the_kernel_before_is_not_a_wait(fmt):
    # behind one row that a single CTA takes milliseconds for, so that the next kernel stands beside it:
    # half a millisecond is enough for calls of ten microseconds
    row = normal(1, 1 << 20, seed=1).repeat(1, 96)
    w = quant.quantise(normal(512, 1024, seed=2), fmt)
    x = normal(4, 1024, seed=3)
    a = quant.quantise(x, fmt)
    many = quant.quantise(normal(2304, 1024, seed=4), fmt)  # (with w: CTA pairs)
    calls = [lambda t: quant.product(a, w, timeout_ns=t, static_b=True), lambda t: quant.product(a, w, timeout_ns=t),
             lambda t: quant.linear(x, w, timeout_ns=t, static_b=True), lambda t: quant.linear(x, w, timeout_ns=t),
             lambda t: quant.product(many, many, timeout_ns=t)]
    want = [f(0) for f in calls]
    assert quant.check() == gemm.OK
    for f, c in zip(calls, want):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        quant.quantise(row, "e4m3")
        got = f(500_000)
        end.record()
        assert quant.check() == gemm.OK
        assert begin.elapsed_time(end) > 1.5  # (ms: the row took longer than the limit)
        assert torch.equal(got, c)


@pytest.mark.parametrize("fmt", FOUR)
@pytest.mark.parametrize("cols", [4096, 5120, 6200, 14336, 15000])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_many_rows_are_as_few(fmt, cols, dtype):
    # (the rule for the registers of a row's threads goes by the rows and their width)
    x = normal(1300, cols, seed=cols, to=dtype)
    x[7, 100], x[1299, cols - 1], x[640] = float("nan"), float("inf"), 0
    q = quant.quantise(x, fmt)
    for first in (0, 640, 1280):  # (a scale block's first rows)
        part = quant.quantise(x[first:first + 20], fmt)
        assert torch.equal(q.data[first:first + 20], part.data)
        if fmt == "nvfp4":
            assert torch.equal(q.row_scale[first:first + 20].view(torch.int32), part.row_scale.view(torch.int32))
        across = part.scales.numel() // 512
        assert torch.equal(q.scales.view(-1, across, 32, 16)[first // 128, :, :20, :4], part.scales.view(across, 32, 16)[:, :20, :4])
