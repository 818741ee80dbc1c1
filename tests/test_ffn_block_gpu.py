"""The operators together: the example's stack of blocks, its gradients against
PyTorch's in 64 bits, and single tokens against the whole prompt."""
from __future__ import annotations

import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    import feed_forward_block
    return feed_forward_block


def test_gradients_of_the_stack(example):
    """Every parameter's gradient within a few bf16 roundings of autograd in 64 bits
    (each of the stack's nine stored tensors per block rounds to 2^-9 relative)."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    blocks = [example.Block(256, 320, gen) for _ in range(2)]
    x = torch.randn((200, 256), generator=gen, device="cuda").bfloat16()
    ds = torch.randn((200, 256), generator=gen, device="cuda").bfloat16()
    kept = []
    out = example.forward(blocks, x, kept)
    grads = example.backward(blocks, kept, ds)

    params = [[p.double().requires_grad_() for p in b.parameters()] for b in blocks]

    def rms(v, w):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * w

    s = x.double()
    for w_in, w_out, norm_in, norm_out, scale in params:
        g, u = (rms(s, norm_in) @ w_in.t()).split(320, 1)
        s = s + scale * rms((torch.nn.functional.silu(g) * u) @ w_out.t(), norm_out)
    want = torch.autograd.grad(s, [p for ps in params for p in ps], ds.double())
    assert float((out.double() - s.detach()).norm() / s.detach().norm()) < 6 * 2 ** -9
    got = [g for gs in grads for g in gs]
    assert len(got) == len(want)
    for i, (a, b) in enumerate(zip(got, want)):
        off = float((a.double() - b).norm() / b.norm())
        assert off < 18 * 2 ** -9, (i, off)


def test_training_lowers_the_loss_and_tokens_agree(example):
    losses, off = example.main(["--layers", "2", "--width", "256", "--hidden", "704", "--tokens", "296",
                                "--steps", "12"])
    assert losses[-1] < 0.7 * losses[0]
    assert off < 4 * 2 ** -8
