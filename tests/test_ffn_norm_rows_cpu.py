"""How a norm's rows are cut into copies (csrc/norm.h), walked on the CPU: the pieces
that a bulk copy brings hold nothing outside the array, and with the elements copied one
by one they are the whole row."""
from __future__ import annotations

import os
import subprocess

from dense_gemm_blackwell_sm_gb300 import build as pkg_build

WALK = r"""
#include <algorithm>
#include <cstdio>
#include <vector>
#include "norm.h"
using dgb::RowPieces;

// rows * D elements of `size` bytes, `ld` apart, starting `base` elements past a boundary
static long walk(int size, int base, int M, int D, int ld, int col0, int cols) {
  const int N = 16 / size;
  const bool ends_row = col0 + cols == D;
  const long first = base, last = base + (long)(M - 1) * ld + D;  // the array, in elements from a boundary
  long wrong = 0;
  for (int r = 0; r < M; ++r) {
    const long row = base + (long)r * ld + col0;
    const int shift = (int)(row % N), edge = dgb::rows_at_an_end(ld, N);
    // (a slice that does not start its row has its row's elements before it)
    const bool head = col0 == 0 && base != 0 && r < edge && shift != 0, tail = r >= M - edge;
    const RowPieces p = RowPieces::of(shift, cols, N, ends_row);
    const int begin = p.begin(head) / size, end = p.end(tail) / size;
    std::vector<char> got(shift + cols + N, 0);
    if (begin < end) {
      wrong += row - shift + begin < first || row - shift + end > last;
      for (int e = begin; e < end; ++e) ++got[e];
    }
    // the rest by element, as the kernel takes it
    if (head) {
      for (int e = shift; e < std::min(N, shift + cols); ++e) ++got[e];
      for (int e = std::max({N, end, shift}); e < shift + cols; ++e) ++got[e];
    } else if (tail && p.rest != 0) {
      for (int e = std::max(end, shift); e < end + p.rest; ++e) ++got[e];
    }
    for (int e = shift; e < shift + cols; ++e) wrong += got[e] != 1;
    wrong += ld >= N - 1 && edge != 1;  // rows of a piece and more: the first and the last one alone
  }
  return wrong;
}

int main() {
  long wrong = 0, calls = 0;
  for (int size : {2, 4})
    for (int base = 0; base < 16 / size; ++base)
      for (int M : {1, 2, 3, 9, 20})
        for (int D = 1; D <= 40; ++D)
          for (int gap : {0, 1, 3, 8, 16}) {
            wrong += walk(size, base, M, D, D + gap, 0, D);
            ++calls;
          }
  // slices of wide rows (the last one is longer than a piece)
  for (int D : {41, 47, 48, 61})
    for (int gap : {0, 5}) {
      wrong += walk(2, 0, 5, D, D + gap, 0, 32) + walk(2, 0, 5, D, D + gap, 32, D - 32);
      ++calls;
    }
  std::printf("%ld %ld\n", wrong, calls);
}
"""


def test_row_copies_stay_inside_the_array(tmp_path):
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(WALK)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(pkg_build.nvcc())))
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", pkg_build.INCLUDE, "-I", pkg_build.CSRC, "-isystem",
                    os.path.join(cuda, "include"), str(src), "-o", str(exe)], check=True)
    wrong, calls = map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split())
    assert calls > 4000 and wrong == 0
