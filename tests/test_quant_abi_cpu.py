"""include/quant.h without a GPU: every declared function is exported, the binding's
structures match the header, sizes are as documented, and bad arguments are refused before
any device is touched."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

from oracle import quant as ref
from dense_gemm_blackwell_sm_gb300 import build as pkg_build
from dense_gemm_blackwell_sm_gb300 import ffn, gemm, quant

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000  # an address that is never read
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return quant.load()


def test_every_declared_symbol_is_exported(lib):
    text = open(os.path.join(ROOT, "include", "quant.h")).read()
    names = re.findall(r"GEMM_API\s+[\w\s\*]+?\b(quant_\w+)\s*\(", text)
    assert len(names) == 11
    for n in names:
        assert hasattr(lib, n), n


def test_structures_match_the_header(tmp_path):
    structs = {"quant_rows_t": quant.RowsArgs, "quant_norm_t": quant.NormArgs, "quant_product_t": quant.ProductArgs,
               "quant_linear_t": quant.LinearArgs}
    lines = ["#include <cstddef>", "#include <cstdio>", '#include "quant.h"', "int main() {"]
    want = []
    for c, py in structs.items():
        lines.append('std::printf("%%zu\\n", sizeof(%s));' % c)
        want.append(ctypes.sizeof(py))
        for name, _ in py._fields_:
            lines.append('std::printf("%%zu\\n", offsetof(%s, %s));' % (c, name))
            want.append(getattr(py, name).offset)
    src, exe = tmp_path / "sizes.cpp", tmp_path / "sizes"
    src.write_text("\n".join(lines + ["}"]))
    subprocess.run(["g++", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in got] == want


@pytest.mark.parametrize("rows,cols", [(0, 0), (1, 1), (1, 32), (127, 33), (128, 64), (129, 4097), (5, 0)])
def test_sizes(lib, rows, cols):
    assert quant.width(cols) == ref.width(cols)
    for fmt, code in quant.FORMATS.items():
        o = ref.quantise(np.zeros((max(rows, 1), cols)), fmt)
        assert lib.quant_row_bytes(cols, code) == o.codes.shape[1] // (1 if "e4m3" in fmt else 2)
        want = 0 if o.scales is None or rows == 0 else ref.tile(o.scales, rows).size
        assert quant.scale_bytes(rows, cols, fmt) == want


def test_sizes_refused(lib):
    assert lib.quant_width(-1) == -1 and lib.quant_width(BIG - 32) == -1 and lib.quant_width(BIG - 33) == BIG - 32
    assert lib.quant_row_bytes(5, 4) == -1 and lib.quant_row_bytes(-1, 0) == -1
    assert lib.quant_scale_bytes(-1, 5, 1) == -1 and lib.quant_scale_bytes(BIG, 5, 1) == -1
    assert lib.quant_scale_bytes(5, 5, -1) == -1


def rows_args(**kw):
    a = dict(rows=8, cols=64, dtype=ffn.BF16, format=quant.NVFP4, x=P, data=P, scales=P, row_scale=P)
    a.update(kw)
    return quant.RowsArgs(**a)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), gemm.ERR_UNSUPPORTED_DTYPE), (dict(format=4), gemm.ERR_UNSUPPORTED_DTYPE),
    (dict(format=-1), gemm.ERR_UNSUPPORTED_DTYPE), (dict(transpose=2), gemm.ERR_INVALID_ARG),
    (dict(rows=-1), gemm.ERR_INVALID_ARG), (dict(cols=-1), gemm.ERR_INVALID_ARG), (dict(rows=BIG), gemm.ERR_INVALID_ARG),
    (dict(cols=BIG - 32), gemm.ERR_INVALID_ARG), (dict(ld_x=63), gemm.ERR_INVALID_ARG),
    (dict(rows=BIG - 64, cols=BIG - 64, transpose=1), gemm.ERR_UNSUPPORTED_SHAPE),
    (dict(ld_data=16), gemm.ERR_INVALID_ARG), (dict(ld_data=40), gemm.ERR_MISALIGNED), (dict(x=0), gemm.ERR_INVALID_ARG),
    (dict(data=0), gemm.ERR_INVALID_ARG), (dict(scales=0), gemm.ERR_INVALID_ARG), (dict(row_scale=0), gemm.ERR_INVALID_ARG),
    (dict(format=quant.MXFP4), gemm.ERR_INVALID_ARG), (dict(format=quant.E4M3), gemm.ERR_INVALID_ARG),
    (dict(data=P + 8), gemm.ERR_MISALIGNED), (dict(scales=P + 8), gemm.ERR_MISALIGNED),
    (dict(row_scale=P + 2), gemm.ERR_MISALIGNED), (dict(x=P + 1), gemm.ERR_MISALIGNED),
    (dict(workspace=P + 8), gemm.ERR_MISALIGNED), (dict(transpose=1), gemm.ERR_INVALID_ARG),  # (no workspace)
    (dict(rows=0), gemm.OK), (dict(cols=0, transpose=1), gemm.OK)])
def test_rows_refusals(lib, change, status):
    assert lib.quant_rows(ctypes.byref(rows_args(**change)), None) == status


def test_rows_workspace(lib):
    size = lambda **kw: lib.quant_rows_workspace(ctypes.byref(rows_args(**kw)))  # noqa: E731
    assert size() == 0 and size(transpose=1) >= 4 * 64 and size(transpose=1, format=quant.MXFP4) == 0
    assert size(transpose=1, cols=0) == 0 and size(rows=-1) == -1 and lib.quant_rows_workspace(None) == -1


def norm_args(**kw):
    a = dict(M=8, D=64, dtype=ffn.BF16, param_dtype=ffn.F32, format=quant.E4M3, eps=1e-6, residual_scale=1,
             branch_scale=1, y=P, data=P, row_scale=P)
    a.update(kw)
    return quant.NormArgs(**a)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), gemm.ERR_UNSUPPORTED_DTYPE), (dict(format=4), gemm.ERR_UNSUPPORTED_DTYPE),
    (dict(param_dtype=ffn.F16), gemm.ERR_UNSUPPORTED_DTYPE), (dict(M=-1), gemm.ERR_INVALID_ARG),
    (dict(D=0), gemm.ERR_INVALID_ARG), (dict(D=32769), gemm.ERR_UNSUPPORTED_SHAPE), (dict(y=0), gemm.ERR_INVALID_ARG),
    (dict(ld_y=63), gemm.ERR_INVALID_ARG), (dict(ld_residual=63), gemm.ERR_INVALID_ARG), (dict(ld_s=-64), gemm.ERR_INVALID_ARG),
    (dict(ld_data=32), gemm.ERR_INVALID_ARG), (dict(ld_data=72), gemm.ERR_MISALIGNED),
    (dict(scales=P), gemm.ERR_INVALID_ARG), (dict(row_scale=0), gemm.ERR_INVALID_ARG), (dict(y=P + 1), gemm.ERR_MISALIGNED),
    (dict(weight=P + 2), gemm.ERR_MISALIGNED), (dict(s=P + 1), gemm.ERR_MISALIGNED), (dict(M=0), gemm.OK)])
def test_norm_refusals(lib, change, status):
    assert lib.quant_norm(ctypes.byref(norm_args(**change)), None) == status


def product_args(**kw):
    a = dict(M=4, N=8, K=64, format=quant.NVFP4, out_dtype=ffn.BF16, a=P, b=P, scales_a=P, scales_b=P, c=P)
    a.update(kw)
    return quant.ProductArgs(**a)


@pytest.mark.parametrize("change,status", [
    (dict(format=quant.E4M3), gemm.ERR_UNSUPPORTED_DTYPE), (dict(format=quant.MXE4M3), gemm.ERR_UNSUPPORTED_DTYPE),
    (dict(out_dtype=ffn.F16), gemm.ERR_UNSUPPORTED_DTYPE), (dict(M=-1), gemm.ERR_INVALID_ARG),
    (dict(N=BIG), gemm.ERR_INVALID_ARG), (dict(K=0), gemm.ERR_INVALID_ARG), (dict(K=48), gemm.ERR_UNSUPPORTED_SHAPE),
    (dict(activation=5), gemm.ERR_INVALID_ARG), (dict(flags=2), gemm.ERR_INVALID_ARG),
    (dict(timeout_ns=-1), gemm.ERR_INVALID_ARG), (dict(a=0), gemm.ERR_INVALID_ARG), (dict(b=0), gemm.ERR_INVALID_ARG),
    (dict(scales_a=0), gemm.ERR_INVALID_ARG), (dict(scales_b=0), gemm.ERR_INVALID_ARG), (dict(c=0), gemm.ERR_INVALID_ARG),
    (dict(ld_a=16), gemm.ERR_INVALID_ARG), (dict(ld_b=40), gemm.ERR_MISALIGNED), (dict(ld_c=7), gemm.ERR_INVALID_ARG),
    (dict(ld_residual=7), gemm.ERR_INVALID_ARG), (dict(a=P + 8), gemm.ERR_MISALIGNED), (dict(b=P + 8), gemm.ERR_MISALIGNED),
    (dict(scales_a=P + 8), gemm.ERR_MISALIGNED), (dict(c=P + 1), gemm.ERR_MISALIGNED), (dict(bias=P + 2), gemm.ERR_MISALIGNED),
    (dict(row_scale_a=P + 2), gemm.ERR_MISALIGNED), (dict(residual=P + 1), gemm.ERR_MISALIGNED),
    (dict(M=0), gemm.OK), (dict(N=0), gemm.OK)])
def test_product_refusals(lib, change, status):
    assert lib.quant_product(ctypes.byref(product_args(**change)), None) == status


def linear_args(**kw):
    a = dict(M=40, N=8, K=64, dtype=ffn.BF16, format=quant.NVFP4, out_dtype=ffn.BF16, x=P, b=P, scales_b=P, c=4 * P, workspace=P)
    a.update(kw)
    return quant.LinearArgs(**a)


@pytest.mark.parametrize("change,status", [
    (dict(format=quant.MXE4M3), gemm.ERR_UNSUPPORTED_DTYPE), (dict(dtype=3), gemm.ERR_UNSUPPORTED_DTYPE),
    (dict(out_dtype=ffn.F16), gemm.ERR_UNSUPPORTED_DTYPE), (dict(M=-1), gemm.ERR_INVALID_ARG),
    (dict(N=BIG), gemm.ERR_INVALID_ARG), (dict(K=-1), gemm.ERR_INVALID_ARG), (dict(K=BIG - 32), gemm.ERR_INVALID_ARG),
    (dict(activation=-1), gemm.ERR_INVALID_ARG), (dict(flags=4), gemm.ERR_INVALID_ARG),
    (dict(timeout_ns=-1), gemm.ERR_INVALID_ARG), (dict(x=0), gemm.ERR_INVALID_ARG), (dict(b=0), gemm.ERR_INVALID_ARG),
    (dict(scales_b=0), gemm.ERR_INVALID_ARG), (dict(c=0), gemm.ERR_INVALID_ARG), (dict(workspace=0), gemm.ERR_INVALID_ARG),
    (dict(ld_x=63), gemm.ERR_INVALID_ARG), (dict(ld_b=16), gemm.ERR_INVALID_ARG), (dict(ld_b=40), gemm.ERR_MISALIGNED),
    (dict(ld_c=7), gemm.ERR_INVALID_ARG), (dict(ld_residual=7), gemm.ERR_INVALID_ARG), (dict(x=P + 1), gemm.ERR_MISALIGNED),
    (dict(b=P + 8), gemm.ERR_MISALIGNED), (dict(scales_b=P + 4), gemm.ERR_MISALIGNED), (dict(c=P + 1), gemm.ERR_MISALIGNED),
    (dict(bias=P + 2), gemm.ERR_MISALIGNED), (dict(row_scale_b=P + 1), gemm.ERR_MISALIGNED),
    (dict(residual=P + 1), gemm.ERR_MISALIGNED), (dict(workspace=P + 16), gemm.ERR_MISALIGNED),
    (dict(M=BIG - 511), gemm.ERR_INVALID_ARG), (dict(M=1 << 30, N=1 << 30), gemm.ERR_UNSUPPORTED_SHAPE),
    # C on x, on its second row, over columns of its rows; beside them and behind them all is well
    (dict(x=P, c=P), gemm.ERR_INVALID_ARG), (dict(c=P + 128, K=64), gemm.ERR_INVALID_ARG),
    (dict(ld_x=96, ld_c=96, c=P + 112), gemm.ERR_INVALID_ARG), (dict(ld_x=96, ld_c=80, c=P + 128), gemm.ERR_INVALID_ARG),
    (dict(ld_x=96, ld_c=96, c=P + 2 * 90), gemm.ERR_INVALID_ARG), (dict(c=P - 16, ld_c=64), gemm.ERR_INVALID_ARG),
    (dict(M=0), gemm.OK), (dict(N=0), gemm.OK)])
def test_linear_refusals(lib, change, status):
    assert lib.quant_linear(ctypes.byref(linear_args(**change)), None) == status


def test_linear_workspace(lib):
    size = lambda **kw: lib.quant_linear_workspace(ctypes.byref(linear_args(**kw)))  # noqa: E731
    # the quantised rows: codes, tiled scales, row scales, each to 256 bytes; none in one kernel
    assert size() == 40 * 32 // 256 * 256 + 512 + 256 and size(format=quant.MXFP4) == 1280 + 512
    assert size(M=16) == 0 and size(M=0) == 0 and size(N=0) == 0 and size(M=-1) == -1
    assert size(M=8, N=14336, K=65536) > 0 and lib.quant_linear_workspace(None) == -1


def test_many_rows_refusals(lib):
    # one refused array refuses all; none is no work
    two = (quant.RowsArgs * 2)(rows_args(rows=0), rows_args(dtype=3))
    assert lib.quant_rows_many(two, 2, None) == gemm.ERR_UNSUPPORTED_DTYPE
    assert lib.quant_rows_many(two, 1, None) == gemm.OK and lib.quant_rows_many(two, 0, None) == gemm.OK
    assert lib.quant_rows_many(two, -1, None) == gemm.ERR_INVALID_ARG
    assert lib.quant_rows_many(None, 0, None) == gemm.ERR_INVALID_ARG


def test_null_arguments(lib):
    for f in (lib.quant_rows, lib.quant_norm, lib.quant_product, lib.quant_linear):
        assert f(None, None) == gemm.ERR_INVALID_ARG
