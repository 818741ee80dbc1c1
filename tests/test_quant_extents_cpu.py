"""Where arrays of the low-precision operands end (csrc/quant_launch.h), on the CPU: kernels load whole
16-byte pieces inside [start, end), so an array of no values has to end where it starts."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

from dense_gemm_blackwell_sm_gb300 import build as pkg_build
from dense_gemm_blackwell_sm_gb300 import ffn, gemm, quant

P = 0x10000  # an address that is never read
BIG = 1 << 31

RULE = r"""
#include <cstdio>
#include "quant_launch.h"

int main() {
  for (long at : {0L, 0x10000L})
    for (long rows : {0L, 1L, 2L, 100L})
      for (long cols : {0L, 1L, 33L})
        for (long ld : {0L, 64L, 4096L})
          for (long elem : {2L, 4L}) {
            const void* x = reinterpret_cast<const void*>(at);
            std::printf("%ld %ld %ld %ld %ld %ld\n", at, rows, cols, ld, elem,
                        (long)reinterpret_cast<intptr_t>(dgb::end_of_rows(x, rows, ld, cols, elem)));
          }
}
"""


def test_ends_of_arrays(tmp_path):
    src, exe = tmp_path / "rule.cpp", tmp_path / "rule"
    src.write_text(RULE)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(pkg_build.nvcc())))
    subprocess.run(["g++", "-std=c++17", "-I", pkg_build.INCLUDE, "-I", pkg_build.CSRC, "-isystem",
                    os.path.join(cuda, "include"), str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()
    assert len(lines) == 2 * 4 * 3 * 3 * 2
    for at, rows, cols, ld, elem, end in (map(int, line.split()) for line in lines):
        last = [at + (r * ld + c) * elem + elem for r in range(rows) for c in range(cols)]
        assert end == (max(last) if last else at) or (ld < cols and rows > 1)  # (a pitch below a row is refused)


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return quant.load()


# a pitch and a number of rows that no memory has: refused before a size is computed from them
HUGE = dict(rows=BIG - 64, cols=4, ld_x=BIG - 1)


@pytest.mark.parametrize("dtype", [ffn.F16, ffn.F32])
def test_arrays_past_every_memory_are_refused(lib, dtype):
    a = quant.RowsArgs(**HUGE, dtype=dtype, format=quant.MXFP4, x=P, data=P, scales=P)
    assert lib.quant_rows(ctypes.byref(a), None) == gemm.ERR_INVALID_ARG
    a.transpose = 1
    assert lib.quant_rows(ctypes.byref(a), None) == gemm.ERR_INVALID_ARG
    for ld in ("ld_y", "ld_residual", "ld_s"):
        n = quant.NormArgs(M=BIG - 64, D=4, dtype=dtype, param_dtype=ffn.F32, format=quant.MXFP4, eps=1e-6, y=P,
                           residual=P, s=P, data=P, scales=P, **{ld: BIG - 1})
        assert lib.quant_norm(ctypes.byref(n), None) == gemm.ERR_INVALID_ARG
    for ld in ("ld_c", "ld_residual"):
        p = quant.ProductArgs(M=BIG - 512, N=4, K=64, format=quant.MXFP4, out_dtype=ffn.F32, a=P, b=P, scales_a=P,
                              scales_b=P, c=P, residual=P, **{ld: BIG - 1})
        assert lib.quant_product(ctypes.byref(p), None) == gemm.ERR_INVALID_ARG
    for ld in ("ld_x", "ld_c", "ld_residual"):
        m = quant.LinearArgs(M=BIG - 512, N=4, K=4, dtype=dtype, format=quant.MXFP4, out_dtype=ffn.F32, x=P, b=P, scales_b=P,
                             c=4 * P, residual=P, workspace=P, **{ld: BIG - 1})
        assert lib.quant_linear(ctypes.byref(m), None) == gemm.ERR_INVALID_ARG
