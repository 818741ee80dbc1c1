"""A stack of gated feed-forward blocks trained for a few steps, then run token by
token, with this library's operators alone:

    s, n = block_norm(y, s, ...)          norm after the last block, gate, residual, norm before this one
    h    = gated(n, w_in)                 both projections, activation and product in one kernel
    y    = matmul(h, w_out)               down projection

and the same backwards (tokens, width and hidden width are multiples of 8, since each is
a reduction of `matmul` there).  The blocks learn to reproduce a fixed random stack's output.

    python examples/feed_forward_block.py [--layers 4 --width 1024 --hidden 2752 --tokens 2048 --steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from dense_gemm_blackwell_sm_gb300 import ffn, gemm  # noqa: E402


class Block:
    """One block's parameters: bf16 weights, fp32 norm weights and layer scale."""

    def __init__(self, width, hidden, gen):
        def normal(*shape, std):
            return (torch.randn(shape, generator=gen, device="cuda") * std).bfloat16()

        self.w_in = normal(2 * hidden, width, std=width ** -0.5)   # gate rows, then up rows
        self.w_out = normal(width, hidden, std=hidden ** -0.5)
        self.norm_in = torch.ones(width, device="cuda")            # before the block
        self.norm_out = torch.ones(width, device="cuda")           # after it
        self.scale = torch.full((width,), 0.5, device="cuda")      # layer scale

    def parameters(self):
        return [self.w_in, self.w_out, self.norm_in, self.norm_out, self.scale]


def forward(blocks, x, keep=None):
    """The stream after the last block; with ``keep`` (a list) what the backward pass needs is left there."""
    s, n = ffn.block_norm(x, pre_weight=blocks[0].norm_in)  # the first norm: the stream is x itself
    for i, b in enumerate(blocks):
        following = blocks[i + 1].norm_in if i + 1 < len(blocks) else None
        made = ffn.gated(n, b.w_in, act="silu", save=keep is not None)
        h, gu = made if keep is not None else (made, None)
        y = gemm.matmul(h, b.w_out, out_dtype=torch.bfloat16)
        if keep is not None:
            keep.append((s, n, gu, h, y))
        s, n = ffn.block_norm(y, s, post_norm=True, post_weight=b.norm_out, gate=b.scale,
                              pre_norm=following is not None, pre_weight=following)
        if keep is not None:
            keep[-1] += (s,)
    return s


def backward(blocks, kept, ds):
    """Gradients of every block's parameters, in their order."""
    grads, dn = [None] * len(blocks), None
    for i in reversed(range(len(blocks))):
        b, (s, n, gu, h, y, s_next) = blocks[i], kept[i]
        following = blocks[i + 1].norm_in if i + 1 < len(blocks) else None
        g = ffn.block_norm_backward(ds, dn, y, s_next, post_norm=True, post_weight=b.norm_out, gate=b.scale,
                                    pre_norm=following is not None, pre_weight=following)
        if following is not None:
            grads[i + 1][2] = g.dpre_weight
        dh = gemm.matmul(g.dy, b.w_out.t(), out_dtype=torch.bfloat16)       # dy w_out
        dw_out = gemm.matmul(g.dy.t(), h.t(), out_dtype=torch.bfloat16)     # dy^T h
        dn, dw_in = ffn.gated_backward(dh, n, b.w_in, gu=gu, act="silu")
        ds = g.dresidual
        grads[i] = [dw_in, dw_out, None, g.dpost_weight, g.dgate]
    g = ffn.block_norm_backward(ds, dn, None, kept[0][0], pre_weight=blocks[0].norm_in, need_dy=False)
    grads[0][2] = g.dpre_weight
    return grads


def train(blocks, x, target, steps, rate):
    losses = []
    for _ in range(steps):
        kept = []
        out = forward(blocks, x, kept)
        off = out.float() - target.float()
        losses.append(float((off * off).mean()))
        grads = backward(blocks, kept, (off * (2.0 / off.numel() * 1024)).bfloat16())  # loss scaled by 1024
        for b, gs in zip(blocks, grads):
            for p, g in zip(b.parameters(), gs):
                g = g.float() / 1024
                p.sub_((rate * g / (g.square().mean().sqrt() + 1e-12) * p.float().square().mean().sqrt()).to(p.dtype))
    return losses


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2752)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(0)
    teacher = [Block(a.width, a.hidden, gen) for _ in range(a.layers)]
    blocks = [Block(a.width, a.hidden, gen) for _ in range(a.layers)]
    x = torch.randn((a.tokens, a.width), generator=gen, device="cuda").bfloat16()
    losses = train(blocks, x, forward(teacher, x), a.steps, 0.02)
    print("loss %.4f -> %.4f in %d steps" % (losses[0], losses[-1], a.steps))
    whole = forward(blocks, x[:16])
    single = torch.cat([forward(blocks, x[i:i + 1]) for i in range(16)])
    off = float((whole.float() - single.float()).abs().max() / whole.float().abs().max())
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(100):
        forward(blocks, x[:1])
    torch.cuda.synchronize()
    print("one token at a time: off by %.2g of the largest value, %.1f us per token and block"
          % (off, (time.perf_counter() - t0) * 1e4 / a.layers))
    assert ffn.check() == gemm.OK and gemm.gemm_check() == gemm.OK
    return losses, off


if __name__ == "__main__":
    main()
