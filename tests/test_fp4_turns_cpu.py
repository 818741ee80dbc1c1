"""How the accumulators of the 4-bit product's CTA pairs go from tile to tile (csrc/fp4_turns.h): every
order of the MMAs and the epilogue's arrivals is walked on the CPU, with the phases of the barriers
as the hardware keeps them."""
from __future__ import annotations

import os
import subprocess

import pytest

from dense_gemm_blackwell_sm_gb300 import build as pkg_build

TILES = 9
WARPS = 3  # (of the epilogue: each arrives for itself, and what counts is that they are several)

RULE = r"""
#include <cstdio>
#include "fp4_turns.h"

int main() {
  for (unsigned n = 0; n < TILES; ++n) std::printf("%u %u\n", dgb::fp4_turn(n), dgb::fp4_empty_parity(n));
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    at = tmp_path_factory.mktemp("turns")
    src, exe = at / "rule.cpp", at / "rule"
    src.write_text(RULE)
    subprocess.run(["g++", "-std=c++17", "-DTILES=%d" % TILES, "-I", pkg_build.CSRC, str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()
    return [tuple(map(int, line.split())) for line in lines]


def walk(parities, own=None):
    """All orders in which a cluster's tiles can go, tile n waiting for the phase `parities[n]` of the
    barrier that every warp arrives on when it has read its common columns; with `own` also, from tile 2
    on, for the phase own[n] of another, arrived on when it has read the tile's own columns.  Returns the
    orders that stop and the tiles whose MMAs begin too early.

    A barrier is the arrivals of its present phase and how many phases have ended; a wait for a parity
    passes where the phase before the present one has it (none yet: parity one)."""
    tiles = len(parities)
    # MMA: its tile and whether it has passed the first wait; warps: 3 * tile + what they have done of it
    # (waited for the sums, read the common columns, read the own ones); the two barriers
    start = ((0, 0), (0,) * WARPS, (0, 0), (0, 0))
    seen, todo, stopped, early = {start}, [start], [], set()
    read_common, read_own = 2, 3

    def arrive(bar):
        count, phase = bar
        return (0, phase + 1) if count + 1 == WARPS else (count + 1, phase)

    def passes(bar, parity):
        return (bar[1] & 1) != parity

    while todo:
        state = todo.pop()
        (tile, half), warps, empty, others = state
        after = []
        if tile < tiles:
            if half == 0 and passes(empty, parities[tile]):
                after.append(((tile, 1), warps, empty, others))
            if half == 1 and (own is None or tile < 2 or passes(others, own[tile])):
                # its MMAs write now: tile - 1's common columns and tile - 2's own ones are to be read
                if min(warps) < 3 * (tile - 1) + read_common or min(warps) < 3 * (tile - 2) + read_own:
                    early.add(tile)
                after.append(((tile + 1, 0), warps, empty, others))
        for i, w in enumerate(warps):
            n, done = divmod(w, 3)
            if n == tiles or (done == 0 and tile <= n):  # (a tile's sums are complete when the MMA is past it)
                continue
            moved = warps[:i] + (w + 1,) + warps[i + 1:]
            after.append(((tile, half), moved, arrive(empty) if done + 1 == read_common else empty,
                          arrive(others) if done + 1 == read_own else others))
        if not after and (tile < tiles or min(warps) < 3 * tiles):
            stopped.append(state)
        for s in after:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return stopped, early


def test_no_order_stops_or_writes_too_early(rule):
    assert [t[0] for t in rule] == [n % 2 for n in range(TILES)]
    stopped, early = walk([t[1] for t in rule])
    assert not stopped and not early


def test_the_walk_sees_a_phase_that_is_missed(rule):
    # a second barrier for the own columns, as there was: it may complete for tile n - 1 as well before
    # tile n's wait for tile n - 2 looks at it, and then only tile n itself ends the phase waited for
    stopped, early = walk([t[1] for t in rule], own=[n & 1 for n in range(TILES)])
    assert stopped and not early


def test_the_walk_sees_columns_written_too_early(rule):
    # waits that are a phase behind
    assert walk([1, 1] + [t[1] for t in rule][1:-1])[1]
