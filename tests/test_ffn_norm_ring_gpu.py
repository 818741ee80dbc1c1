"""The block norms at the sizes of prompts, where rows come through a ring in shared
memory: every combination of parts, in place, with pitches and off their boundary, with
values that are not finite; element by element against the 64-bit definitions."""
from __future__ import annotations

import pytest
import torch

from dense_gemm_blackwell_sm_gb300 import ffn, gemm
from test_ffn_gpu import DEV, assert_within, check_norm, norm_inputs, ref_norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert ffn.check() == gemm.OK


# a warp per row with 1, 2 and 4 vectors per lane, a CTA per row with 2 and (RMS) 4; even and odd widths
RING = [(5000, 200, "bf16"), (5001, 31, "f16"), (5000, 255, "f16"), (5000, 500, "bf16"), (5003, 1000, "bf16"),
        (5000, 907, "f16"), (3000, 1031, "bf16"), (1600, 4097, "f16"), (1300, 8200, "bf16"), (1301, 8201, "f16"),
        (5000, 100, "f32"), (5000, 251, "f32"), (5000, 509, "f32"), (3000, 1031, "f32"), (1300, 5001, "f32")]

# post, pre, residual, need_s
PARTS = [(True, True, True, True), (True, True, False, True), (True, False, True, True), (False, True, True, True),
         (False, False, True, True), (True, True, True, False), (False, True, False, True)]


@pytest.mark.parametrize("M,D,dtype", RING)
@pytest.mark.parametrize("parts", range(len(PARTS)))
def test_ring_parts(M, D, dtype, parts):
    post, pre, residual, need_s = PARTS[parts]
    divisors = [g for g in (1, 5, M // 4, 3, M) if M % g == 0]
    for kind in ("rms", "layer") if parts < 2 else (("rms", "layer")[(parts + D) % 2],):
        groups = divisors[(parts + D + (kind == "rms")) % len(divisors)]
        t, p = norm_inputs(M, D, dtype, "f32" if parts % 2 else dtype, kind, groups, M + D + parts)
        if not post:
            p["post_weight"] = p["post_bias"] = None
        if not pre:
            p["pre_weight"] = p["pre_bias"] = None
        if not residual:
            t["residual"] = None
        kw = dict(kind=kind, eps=1e-6, residual_scale=0.5, branch_scale=-1.5)
        s, n = ffn.block_norm(t["y"], t["residual"], post_norm=post, pre_norm=pre, need_s=need_s, **p, **kw)
        want_s, want_n = ref_norm(t, p, dtype, post=post, pre=pre, **kw)
        assert (s is None) == (not need_s) and (n is None) == (not pre)
        if need_s:
            assert_within(s, want_s, "s")
        if pre:
            assert_within(n, want_n, "n")


def rows_at(v, off, pitch, fill):
    """A copy of v whose rows lie `pitch` apart, `off` elements past a boundary, amid `fill`."""
    M, D = v.shape
    flat = torch.full((off + M * pitch + 16,), fill, dtype=v.dtype, device=DEV)
    view = flat[off:off + M * pitch].view(M, pitch)[:, :D] if pitch > D else flat[off:off + M * D].view(M, D)
    view.copy_(v)
    return flat, view


@pytest.mark.parametrize("M,D,dtype", [r for r in RING if r[1] in (31, 255, 500, 1000, 1031, 4097, 8201, 251, 5001)])
@pytest.mark.parametrize("off,gap", [(0, 0), (1, 0), (3, 0), (0, 8), (1, 16), (0, 5)])
def test_ring_in_place_pitched_and_unaligned(M, D, dtype, off, gap):
    """NaN around the inputs, guards around the outputs: nothing outside is read into a result or written."""
    kind = "layer" if (D + off) % 2 else "rms"
    t, p = norm_inputs(M, D, dtype, "f32", kind, 1 if off else 5 if M % 5 == 0 else 1, D + off)
    kw = dict(kind=kind, eps=1e-6)
    want_s, want_n = ref_norm(t, p, dtype, post=True, pre=True, **kw)
    _, y = rows_at(t["y"], off, D + gap, float("nan"))
    _, res = rows_at(t["residual"], off, D + gap, float("nan"))
    flat_s, s = rows_at(torch.zeros_like(t["y"]), off, D + gap, 7.0)
    flat_n, n = rows_at(torch.zeros_like(t["y"]), off, D + gap, 7.0)
    ffn.block_norm(y, res, post_norm=True, s=s, n=n, **p, **kw)
    assert_within(s, want_s, "s")
    assert_within(n, want_n, "n")
    for flat, view in ((flat_s, s), (flat_n, n)):
        inside = torch.zeros(flat.shape, dtype=torch.bool, device=DEV)
        inside[off:off + M * (D + gap)].view(M, D + gap)[:, :D] = True
        assert bool((flat[~inside] == 7).all())
    s2, n2 = ffn.block_norm(y, res, post_norm=True, s=res, n=y, **p, **kw)
    assert s2 is res and n2 is y and torch.equal(res, s) and torch.equal(y, n)


@pytest.mark.parametrize("M,D,dtype,kind", [(2500, 255, "bf16", "layer"), (5000, 31, "f16", "rms"), (600, 1031, "f32", "rms"),
                                            (900, 4100, "bf16", "rms"), (700, 4601, "f16", "layer"), (300, 8200, "f32", "layer"),
                                            (40, 3, "bf16", "rms"), (7, 5, "f32", "layer")])
def test_gradient_pitched_and_unaligned(M, D, dtype, kind):
    """Many rows (and rows shorter than 16 bytes) of every pitch and offset: the same bits."""
    t, p = norm_inputs(M, D, dtype, "f32", kind, 1, M + D)
    s, _, want = check_norm(t, p, dtype, kind)
    for offs, gaps in (((0, 0, 0, 0), (8, 16, 0, 24)), ((1, 0, 2, 3), (0, 1, 3, 0)), ((0, 5, 0, 0), (8, 0, 0, 5))):
        moved = [rows_at(v, o, D + g, float("nan"))[1]
                 for v, o, g in zip((t["ds"], t["dn"], t["y"], s), offs, gaps)]
        got = ffn.block_norm_backward(*moved, post_norm=True, kind=kind, **p)
        for name, a, b in zip(got._fields, got, want):
            assert (a is None) == (b is None) and (a is None or torch.equal(a, b)), (name, offs, gaps)


@pytest.mark.parametrize("M,D,dtype", [(5000, 255, "f16"), (3000, 1031, "bf16"), (5000, 1000, "bf16")])
def test_ring_values_that_are_not_finite_stay_in_their_row(M, D, dtype):
    t, p = norm_inputs(M, D, dtype, "f32", "rms", 1, 1)
    s, n = ffn.block_norm(t["y"], t["residual"], post_norm=True, **p)
    rows = torch.tensor([0, 1, 777, M // 2, M - 2, M - 1], device=DEV)
    for i, r in enumerate(rows.tolist()):
        t["y"][r, (0, D - 1, 17)[i % 3]] = (float("inf"), float("nan"))[i % 2]
    s2, n2 = ffn.block_norm(t["y"], t["residual"], post_norm=True, **p)
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[rows] = False
    assert torch.equal(s2[keep], s[keep]) and torch.equal(n2[keep], n[keep])
    assert bool(n2[rows].isnan().any(1).all())


def test_ring_in_a_graph_and_on_another_stream():
    t, p = norm_inputs(5000, 255, "bf16", "f32", "layer", 5, 6)
    run = lambda **kw: ffn.block_norm(t["y"], t["residual"], post_norm=True, kind="layer", **p, **kw)  # noqa: E731
    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = run(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for g in got:
        g.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
