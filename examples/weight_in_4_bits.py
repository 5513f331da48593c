"""A linear layer's weight, from its updates to the 4 bits that serve it.

The layer is trained with its products in 8 bits (fp8.linear); each step's update is the
momentum's polar factor (Gemm.orthogonalize), so that all directions of the weight move
alike.  The trained weight is then quantised once to nvfp4 and to mxfp4 and serves rows
(fp4.linear).

    python examples/weight_in_4_bits.py [--hidden 1024] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from dense_gemm_tmem_gb300 import fp4, fp8
from dense_gemm_tmem_gb300.gemm import Gemm


def train(g: Gemm, hidden: int, steps: int, rows: int = 512, rate: float = 0.05,
          momentum: float = 0.9):
    """Fits W (2 hidden x hidden) to a random linear map; returns the losses and the weight."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    target = torch.randn(2 * hidden, hidden, generator=gen, device="cuda") * hidden ** -0.5
    w = torch.zeros_like(target, requires_grad=True)
    m = torch.zeros_like(target)
    losses = []
    for _ in range(steps):
        x = torch.randn(rows, hidden, generator=gen, device="cuda").bfloat16()
        loss = (fp8.linear(g, x, w).float() - x.float() @ target.t()).square().mean()
        loss.backward()
        with torch.no_grad():
            m.mul_(momentum).add_(w.grad)
            w -= rate * g.orthogonalize(m).float()
            w.grad = None
        losses.append(float(loss.detach()))
    return losses, w.detach(), target


def serve(g: Gemm, w: torch.Tensor, format: str):
    """Rows through the 4-bit weight, against the weight itself: relative error."""
    wq = g.fp4_quantize(w, format)  # once
    x = torch.randn(8, w.shape[1], device="cuda").bfloat16()
    y = torch.cat([fp4.linear(g, x[i:i + 1], wq) for i in range(8)]).float()
    want = x.float() @ w.t()
    return float((y - want).norm() / want.norm())


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    g = Gemm(torch.device("cuda", 0))
    torch.manual_seed(0)
    losses, w, _ = train(g, a.hidden, a.steps)
    print("training: mean square error %.4f -> %.4f in %d steps" % (losses[0], losses[-1], a.steps))
    off = {f: serve(g, w, f) for f in ("nvfp4", "mxfp4")}
    for f, e in off.items():
        print("serving in %s (weight and activations): relative error %.3f" % (f, e))
    g.status()
    g.close()
    return losses, off


if __name__ == "__main__":
    main()
