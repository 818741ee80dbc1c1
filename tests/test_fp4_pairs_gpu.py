"""The 4-bit product on CTA pairs (csrc/kernels_fp4_pair.cu), where a cluster takes several tiles one
after another: both accumulators, their hand-over, scales of later tiles."""
from __future__ import annotations

import numpy as np
import pytest
import torch

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


def codes(rows, cols, fmt, seed):
    """A random operand (every code, scales of 1/2, 1 and 2) for the oracle."""
    rng = np.random.default_rng(seed)
    w = ref.width(cols)
    c = rng.integers(0, 16, (rows, w)).astype(np.uint8)
    c[:, cols:] = 0
    one, step = (56, 8) if fmt == "nvfp4" else (127, 1)
    s = one + step * rng.integers(-1, 2, (rows, w // ref.BLOCK[fmt]))
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
def test_several_tiles_of_a_cluster(shape, fmt, out):
    M, N, K = shape
    a, b = codes(M, K, fmt, 1), codes(N, K, fmt, 2)
    qa, qb, want = device(a), device(b), times(a, b).to(OUT[out])
    for _ in range(3):
        c = quant.product(qa, qb, out_dtype=OUT[out])
        assert quant.check() == gemm.OK
        assert torch.equal(c, want), torch.nonzero(c != want)[:3]


@pytest.mark.parametrize("fmt", FOUR)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("K", [96, 2080])
def test_a_wait_that_runs_out_ends_every_role(fmt, out, K):
    # each CTA's first copy is left out: what waits for it gives up, then what waits for that, over
    # several tiles; the calls behind it are whole
    M, N = 4352, 4200
    a, b = codes(M, K, fmt, 3), codes(N, K, fmt, 4)
    qa, qb, want = device(a), device(b), times(a, b).to(OUT[out])
    quant.product(qa, qb, out_dtype=OUT[out], timeout_ns=20_000_000, debug_flags=quant.DEBUG_SKIP_ONE_LOAD)
    c = quant.product(qa, qb, out_dtype=OUT[out])
    assert quant.check() == gemm.ERR_DEVICE_TIMEOUT
    assert torch.equal(c, want) and quant.check() == gemm.OK
    assert torch.equal(quant.product(qa, qb, out_dtype=OUT[out]), want) and quant.check() == gemm.OK
