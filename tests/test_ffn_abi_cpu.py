"""include/ffn.h without a GPU: every declared function is exported, the binding's
structures match the header, and bad arguments are refused before any device is
touched."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import pytest
import torch

from dense_gemm_blackwell_sm_gb300 import build as pkg_build
from dense_gemm_blackwell_sm_gb300 import ffn, gemm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000  # an address that is never read


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return ffn.load()


def test_every_declared_symbol_is_exported(lib):
    text = open(os.path.join(ROOT, "include", "ffn.h")).read()
    names = re.findall(r"GEMM_API\s+[\w\s\*]+?\b(ffn_\w+)\s*\(", text)
    assert len(names) >= 6
    for n in names:
        assert hasattr(lib, n), n


def test_structures_match_the_header(tmp_path):
    structs = {"ffn_gated_t": ffn.GatedArgs, "ffn_gated_grad_t": ffn.GatedGradArgs, "ffn_norm_t": ffn.NormArgs,
               "ffn_norm_grad_t": ffn.NormGradArgs}
    lines = ["#include <cstddef>", "#include <cstdio>", '#include "ffn.h"', "int main() {"]
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


def gated_args(**kw):
    a = dict(M=4, F=16, K=64, dtype=ffn.BF16, activation=gemm.ACT_SILU, x=P, w=P, h=P)
    a.update(kw)
    return ffn.GatedArgs(**a)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=ffn.F32), gemm.ERR_UNSUPPORTED_DTYPE), (dict(dtype=7), gemm.ERR_UNSUPPORTED_DTYPE),
    (dict(M=-1), gemm.ERR_INVALID_ARG), (dict(F=0), gemm.ERR_INVALID_ARG), (dict(K=0), gemm.ERR_INVALID_ARG),
    (dict(F=1 << 30), gemm.ERR_INVALID_ARG), (dict(activation=5), gemm.ERR_INVALID_ARG),
    (dict(activation=-1), gemm.ERR_INVALID_ARG), (dict(timeout_ns=-1), gemm.ERR_INVALID_ARG),
    (dict(K=60), gemm.ERR_UNSUPPORTED_SHAPE), (dict(x=0), gemm.ERR_INVALID_ARG), (dict(w=0), gemm.ERR_INVALID_ARG),
    (dict(h=0), gemm.ERR_INVALID_ARG), (dict(x=P + 8), gemm.ERR_MISALIGNED), (dict(w=P + 2), gemm.ERR_MISALIGNED),
    (dict(h=P + 1), gemm.ERR_MISALIGNED), (dict(gu=P + 1), gemm.ERR_MISALIGNED),
    (dict(ld_x=63), gemm.ERR_INVALID_ARG), (dict(ld_x=68), gemm.ERR_MISALIGNED),
    (dict(ld_w=68), gemm.ERR_MISALIGNED), (dict(ld_h=15), gemm.ERR_INVALID_ARG),
    (dict(ld_gu=31), gemm.ERR_INVALID_ARG), (dict(ld_h=-16), gemm.ERR_INVALID_ARG), (dict(M=0), gemm.OK)])
def test_gated_refusals(lib, change, status):
    assert lib.ffn_gated(ctypes.byref(gated_args(**change)), None) == status


def grad_args(**kw):
    a = dict(M=4, F=16, K=64, dtype=ffn.F16, activation=gemm.ACT_RELU, x=P, w=P, gu=P, dh=P, dgu=P, dx=P, dw=P)
    a.update(kw)
    return ffn.GatedGradArgs(**a)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=ffn.F32), gemm.ERR_UNSUPPORTED_DTYPE), (dict(K=12), gemm.ERR_UNSUPPORTED_SHAPE),
    (dict(M=-2), gemm.ERR_INVALID_ARG), (dict(dh=0), gemm.ERR_INVALID_ARG), (dict(dgu=0), gemm.ERR_INVALID_ARG),
    (dict(dgu=P + 8), gemm.ERR_MISALIGNED), (dict(ld_dgu=36), gemm.ERR_MISALIGNED),
    (dict(ld_dgu=24), gemm.ERR_INVALID_ARG), (dict(x=0), gemm.ERR_INVALID_ARG), (dict(w=0), gemm.ERR_INVALID_ARG),
    (dict(gu=0, x=0, dw=0), gemm.ERR_INVALID_ARG), (dict(gu=0, w=0, dx=0), gemm.ERR_INVALID_ARG),
    (dict(gu=P + 1), gemm.ERR_MISALIGNED), (dict(dh=P + 1), gemm.ERR_MISALIGNED),
    (dict(dx=P + 1), gemm.ERR_MISALIGNED), (dict(dw=P + 1), gemm.ERR_MISALIGNED),
    (dict(ld_dx=60), gemm.ERR_INVALID_ARG), (dict(ld_dw=63), gemm.ERR_INVALID_ARG),
    (dict(activation=9), gemm.ERR_INVALID_ARG), (dict(M=0, dw=0), gemm.OK)])
def test_gated_backward_refusals(lib, change, status):
    assert lib.ffn_gated_backward(ctypes.byref(grad_args(**change)), None) == status


def norm_args(**kw):
    a = dict(M=4, D=16, groups=1, dtype=ffn.BF16, param_dtype=ffn.F32, kind=0, flags=3, eps=1e-6, residual_scale=1,
             branch_scale=1, y=P, residual=P, gate=P, post_weight=P, pre_weight=P, s=P, n=P)
    a.update(kw)
    return ffn.NormArgs(**a)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), gemm.ERR_UNSUPPORTED_DTYPE), (dict(param_dtype=ffn.F16), gemm.ERR_UNSUPPORTED_DTYPE),
    (dict(M=-1), gemm.ERR_INVALID_ARG), (dict(D=0), gemm.ERR_INVALID_ARG),
    (dict(D=32769), gemm.ERR_UNSUPPORTED_SHAPE), (dict(kind=2), gemm.ERR_INVALID_ARG),
    (dict(flags=4), gemm.ERR_INVALID_ARG), (dict(groups=3), gemm.ERR_INVALID_ARG),
    (dict(groups=0), gemm.ERR_INVALID_ARG), (dict(groups=8), gemm.ERR_INVALID_ARG), (dict(y=0), gemm.ERR_INVALID_ARG),
    (dict(n=0), gemm.ERR_INVALID_ARG), (dict(flags=1), gemm.ERR_INVALID_ARG),
    (dict(flags=1, n=0, s=0), gemm.ERR_INVALID_ARG), (dict(y=P + 1), gemm.ERR_MISALIGNED),
    (dict(gate=P + 2), gemm.ERR_MISALIGNED), (dict(s=P + 1), gemm.ERR_MISALIGNED), (dict(ld_y=8), gemm.ERR_INVALID_ARG),
    (dict(M=0), gemm.OK)])
def test_norm_refusals(lib, change, status):
    assert lib.ffn_norm(ctypes.byref(norm_args(**change)), None) == status


def norm_grad_args(**kw):
    a = dict(M=4, D=16, groups=1, dtype=ffn.BF16, param_dtype=ffn.F32, kind=1, flags=3, eps=1e-6, residual_scale=1,
             branch_scale=1, ds=P, dn=P, y=P, s=P, gate=P, post_weight=P, pre_weight=P, dresidual=P, dy=P, dgate=P,
             dpost_weight=P, dpre_weight=P, workspace=P)
    a.update(kw)
    return ffn.NormGradArgs(**a)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=-1), gemm.ERR_UNSUPPORTED_DTYPE), (dict(D=1 << 31), gemm.ERR_INVALID_ARG),
    (dict(dn=0), gemm.ERR_INVALID_ARG), (dict(s=0), gemm.ERR_INVALID_ARG), (dict(y=0), gemm.ERR_INVALID_ARG),
    (dict(flags=2), gemm.ERR_INVALID_ARG), (dict(flags=1, dn=0), gemm.ERR_INVALID_ARG),
    (dict(flags=0, ds=0, dn=0, dpost_weight=0, dpre_weight=0), gemm.ERR_INVALID_ARG),
    (dict(workspace=0), gemm.ERR_INVALID_ARG), (dict(workspace=P + 8), gemm.ERR_MISALIGNED),
    (dict(dgate=P + 2), gemm.ERR_MISALIGNED), (dict(ld_dy=15), gemm.ERR_INVALID_ARG),
    (dict(M=0, dgate=0, dpost_weight=0, dpre_weight=0), gemm.OK)])
def test_norm_backward_refusals(lib, change, status):
    assert lib.ffn_norm_backward(ctypes.byref(norm_grad_args(**change)), None) == status


def test_gated_backward_workspace(lib):
    """Asked for where few tokens meet a long reduction; then it has to be there."""
    size = lambda **kw: lib.ffn_gated_backward_workspace(ctypes.byref(grad_args(**kw)))  # noqa: E731
    assert lib.ffn_gated_backward_workspace(None) == -1
    assert size(K=12) == -1 and size() == 0 and size(M=0) == 0 and size(M=8192, F=14336, K=4096) == 0
    wide = dict(M=64, F=14336, K=512)
    n = size(**wide)
    assert n > 0 and n % (64 * 512 * 4) == 0 and size(**wide, dx=0) == 0
    assert lib.ffn_gated_backward(ctypes.byref(grad_args(**wide)), None) == gemm.ERR_INVALID_ARG
    assert lib.ffn_gated_backward(ctypes.byref(grad_args(**wide, workspace=P + 16)), None) == gemm.ERR_MISALIGNED


def test_null_arguments_and_workspace(lib):
    for f in (lib.ffn_gated, lib.ffn_gated_backward, lib.ffn_norm, lib.ffn_norm_backward):
        assert f(None, None) == gemm.ERR_INVALID_ARG
    assert lib.ffn_norm_backward_workspace(None) == -1
    assert lib.ffn_norm_backward_workspace(ctypes.byref(norm_grad_args(D=0))) == -1
    assert lib.ffn_norm_backward_workspace(ctypes.byref(norm_grad_args())) > 0
    assert lib.ffn_norm_backward_workspace(
        ctypes.byref(norm_grad_args(dgate=0, dpost_weight=0, dpre_weight=0))) == 0


def test_binding_refuses_cpu_tensors_and_bad_shapes():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ffn.gated(x, w)
    with pytest.raises(ValueError):
        ffn.gated(x, w[:31])
    with pytest.raises(ValueError):
        ffn.gated(x, w[:, :32])
    with pytest.raises(ValueError):
        ffn.gated(x, w.half())
    with pytest.raises(ValueError):
        ffn.gated(x.float(), w.float())
    with pytest.raises(ValueError):
        ffn.gated(x.t().contiguous().t(), w)
    with pytest.raises(ValueError):
        ffn.gated_backward(torch.zeros(4, 15, dtype=torch.bfloat16), x, w)
    with pytest.raises(ValueError, match="CUDA"):
        ffn.block_norm(x, x)
    with pytest.raises(ValueError):
        ffn.block_norm(x, x[:3])
    with pytest.raises(ValueError):
        ffn.block_norm(x, x, post_weight=torch.ones(64))
    with pytest.raises(ValueError):
        ffn.block_norm(x, x, pre_norm=False, pre_weight=torch.ones(64))
    with pytest.raises(ValueError):
        ffn.block_norm(x, x, pre_weight=torch.ones(63))
    with pytest.raises(ValueError):
        ffn.block_norm(x, x, pre_weight=torch.ones(64), gate=torch.ones(64).bfloat16())
    with pytest.raises(ValueError):
        ffn.block_norm(x, x, gate=torch.ones(3, 64))
    with pytest.raises(ValueError):
        ffn.block_norm(x, x, kind="batch")
    with pytest.raises(ValueError):
        ffn.block_norm_backward(None, None, x, x)
    with pytest.raises(ValueError):
        ffn.block_norm_backward(x, None, x, x)


def test_binding_refuses_what_is_no_tensor():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: ffn.gated(x, [1.0]), lambda: ffn.gated(None, x), lambda: ffn.gated_backward(1, x, x),
                 lambda: ffn.block_norm("y"), lambda: ffn.block_norm(x, 3), lambda: ffn.block_norm(x, gate=1.0),
                 lambda: ffn.block_norm_backward(x, x, x, 0), lambda: ffn.block_norm(x, eps="small")):
        with pytest.raises((TypeError, ValueError)):
            call()
