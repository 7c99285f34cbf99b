#!/usr/bin/env python3
"""Trains a minGRU layer and serves it in 8 bits.

    python examples/train_and_serve_8bit.py [--dim 128] [--steps 200]

A layer learns to reproduce a teacher layer on random sequences: the scan and
its backward kernel run in the library, the two projections through torch, and
the AdamW step keeps its states in 8 bits.  The trained weights are then
quantised once and serve a batch of streams: the prompt in one parallel
forward, the rest token by token, on 8-bit products.
"""

from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import scan_linear_rnn_amd as sr  # noqa: E402


def train(teacher, dim, steps, batch, length, generator):
    """Fits (W_in, W_out) to the teacher's outputs; returns them and the losses."""
    W_in = torch.nn.Parameter(torch.randn(dim, 2 * dim, generator=generator).cuda() / dim ** 0.5)
    W_out = torch.nn.Parameter(torch.randn(dim, dim, generator=generator).cuda() / dim ** 0.5)
    opt = sr.AdamW([W_in, W_out], lr=1e-2, weight_decay=0.0, state_bits=8)
    losses = []
    for step in range(steps):
        opt.lr = 1e-2 * min(1.0, 2.0 * (steps - step) / steps)
        x = torch.randn(batch, length, dim, generator=generator).cuda()
        k, p = (x @ W_in).chunk(2, dim=-1)
        y = sr.mingru_scan(k, p) @ W_out
        target = teacher(x)
        loss = (y - target).square().mean() / target.square().mean()
        loss.backward()
        opt.step()
        opt.zero_grad()
        losses.append(loss.detach())
    return W_in.detach(), W_out.detach(), torch.stack(losses).tolist()


def serve(layer, x, prompt):
    """The first ``prompt`` tokens in one forward, the others one at a time."""
    y, h = layer(x[:, :prompt], None, return_next_prev_hidden=True)
    out = [y]
    for t in range(prompt, x.shape[1]):
        y, h = layer(x[:, t], h, return_next_prev_hidden=True)
        out.append(y.unsqueeze(1))
    return torch.cat(out, dim=1)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--dim", type=int, default=128)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--length", type=int, default=128)
    a = ap.parse_args(argv)
    g = torch.Generator()
    g.manual_seed(0)
    teacher = sr.MinGRU(a.dim, generator=g)
    W_in, W_out, losses = train(teacher, a.dim, a.steps, a.batch, a.length, g)
    layer = sr.MinGRU(a.dim, W_in=W_in, W_out=W_out)
    x = torch.randn(a.batch, a.length, a.dim, generator=g).cuda()
    exact = layer(x)
    served = serve(layer.quantized(), x, a.length // 2)
    error = float((served - exact).norm() / exact.norm())
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.4f} after {a.steps} steps with 8-bit optimizer states; "
          f"served in 8 bits within {100 * error:.2f}% of fp32")
    return losses, error


if __name__ == "__main__":
    main()
