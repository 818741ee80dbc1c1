"""The norm with a quantised output at the ends of fp32's range: rows whose sum of squares passes it, and
weights that only the normalised values can be multiplied by."""
from __future__ import annotations

import pytest
import torch

from oracle import quant as ref
from dense_gemm_blackwell_sm_gb300 import gemm, quant
from test_quant_gpu import check_norm, f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FORMATS = ["e4m3", "mxe4m3", "mxfp4", "nvfp4"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def rows(M, D, size, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    return ((1 + torch.rand(M, D, generator=g)) * torch.where(torch.rand(M, D, generator=g) < 0.5, -size, size)).to(dtype)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("param", ["same", "f32"])
@pytest.mark.parametrize("D", [96, 4096, 20000])
def test_a_sum_past_the_range_gives_zeros(fmt, dtype, param, D):
    # (with the weight multiplied in first these rows pass the range too, and zero times that is no zero)
    y = rows(4, D, 1.0, dtype)
    y[1], y[2] = rows(1, D, 1.6e38, dtype)[0], rows(1, D, 3e19, dtype)[0]
    weight = torch.full((D,), 4.0, dtype=dtype if param == "same" else torch.float32)
    _, q = quant.norm_quantise(y.to(DEV), None, weight.to(DEV), format=fmt)
    assert quant.check() == gemm.OK
    keep = [0, 3]
    _, alone = quant.norm_quantise(y[keep].to(DEV), None, weight.to(DEV), format=fmt)
    data, zero = q.data.view(torch.uint8), quant.quantise(torch.zeros(1, D, device=DEV), fmt)
    magnitude = 0x77 if fmt in ("mxfp4", "nvfp4") else 0x7f  # (zeros keep the values' signs)
    assert not (data[1:3] & magnitude).any() and torch.equal(data[keep], alone.data.view(torch.uint8))
    if q.row_scale is not None:
        assert (q.row_scale[1:3] == zero.row_scale).all() and torch.equal(q.row_scale[keep], alone.row_scale)
    if q.scales is not None:
        each = q.scales.view(-1, 32, 4, 4)  # (blocks, row % 32, row / 32, scale)
        assert not each[:, 1:3, 0].any() and torch.equal(each[:, keep, 0], alone.scales.view(-1, 32, 4, 4)[:, :2, 0])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype,param", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                         (torch.float32, torch.float32), (torch.float16, torch.float32)])
@pytest.mark.parametrize("D", [96, 4096, 20000])
@pytest.mark.parametrize("size,weight", [(3e16, 1e25), (1e-16, 1e-24)])
def test_weights_beyond_what_the_rows_can_take(fmt, dtype, param, D, size, weight):
    # |s w| passes fp32's range at either end where n = s w / sqrt(mean s^2) does not
    if dtype == torch.float16:
        size = 3e4 if size > 1 else 1e-4
        weight = 1e35 if size > 1 else 1e-24
    y = rows(3, D, size, dtype)
    w = rows(1, D, weight, param, 2)[0]
    _, q = quant.norm_quantise(y.to(DEV), None, w.to(DEV), format=fmt, eps=0.0)
    assert quant.check() == gemm.OK
    _, (n, en) = ref.norm(f64(y), None, f64(w), "f32", 0.0)
    check_norm(q, n, en, "f32")
