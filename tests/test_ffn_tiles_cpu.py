"""Host rules of the gated projections' tiles (csrc/gated.h), on the CPU."""
from __future__ import annotations

import os
import subprocess

from dense_gemm_blackwell_sm_gb300 import build as pkg_build

RULE = r"""
#include <cstdio>
#include "gated.h"

int main() {
  for (int consumers = 1; consumers <= 2; ++consumers)
    for (int tokens = 1; tokens <= 600; ++tokens) std::printf("%d ", dgb::gated_a_rows(consumers, tokens));
}
"""


def test_rows_of_the_first_operand(tmp_path):
    """What a copy brings is what the kernel's barriers count on: whole operands of 128 rows with two
    consumers; with one, whole 8-row groups that hold every token."""
    src, exe = tmp_path / "rule.cpp", tmp_path / "rule"
    src.write_text(RULE)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(pkg_build.nvcc())))
    subprocess.run(["g++", "-std=c++17", "-I", pkg_build.INCLUDE, "-I", pkg_build.CSRC, "-isystem",
                    os.path.join(cuda, "include"), str(src), "-o", str(exe)], check=True)
    rows = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    one, two = rows[:600], rows[600:]
    assert set(two) == {128}
    for tokens, r in enumerate(one, 1):
        assert r % 8 == 0 and min(tokens, 128) <= r <= 128
    assert one[39] == 40 and one[119] == 120 and one[120] == 128
