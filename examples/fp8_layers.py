"""The block-scaled 8-bit operators as a program uses them together.

A linear layer is trained for a few steps with its three products in 8 bits
(fp8.linear), its weight is then quantised once and serves single rows, and a
mixture-of-experts layer whose weights were quantised once answers a small
batch token by token and all at once.

    python examples/fp8_layers.py [--hidden 1024] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from dense_gemm_tmem_gb300 import fp8
from dense_gemm_tmem_gb300.gemm import COL, Gemm


def train(g: Gemm, hidden: int, steps: int, rows: int = 512):
    """Fits W to a random linear map; returns the losses and the weight."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    target = torch.randn(hidden, hidden, generator=gen, device="cuda") * hidden ** -0.5
    w = torch.zeros(hidden, hidden, device="cuda", requires_grad=True)
    losses = []
    for _ in range(steps):
        x = torch.randn(rows, hidden, generator=gen, device="cuda").bfloat16()
        y = fp8.linear(g, x, w)  # quantises x and W, and in the backward pass dy
        loss = (y.float() - x.float() @ target.t()).square().mean()
        loss.backward()
        with torch.no_grad():
            w -= 0.25 * hidden * w.grad
            w.grad = None
        losses.append(float(loss.detach()))
    return losses, w.detach(), target


def serve(g: Gemm, w: torch.Tensor, target: torch.Tensor):
    """Decode with the trained weight: quantised once, one row at a time."""
    wq = g.fp8_quantize(w, "tile")
    x = torch.randn(4, w.shape[1], device="cuda").bfloat16()
    rows = [g.fp8_matmul(g.fp8_quantize(x[i:i + 1], "row"), wq, b_major=COL) for i in range(4)]
    got, want = torch.cat(rows).float(), x.float() @ target.t()
    return float((got - want).norm() / want.norm())


def experts(g: Gemm, hidden: int, inner: int, count: int = 16, top_k: int = 4, tokens: int = 8):
    """An expert layer on quantised weights: all tokens at once and one by one."""
    def quantised(rows, cols):  # every expert's matrix by the library's quantiser
        parts = [g.fp8_quantize(torch.randn(rows, cols, device="cuda") * cols ** -0.5, "tile")
                 for _ in range(count)]
        pitch = -(-cols // 16) * 16
        data = torch.zeros(count, rows, pitch, dtype=torch.uint8, device="cuda")
        for e, p in enumerate(parts):
            data[e, :, :cols] = p.data.view(torch.uint8)
        return fp8.Fp8Matrix(data[:, :, :cols], torch.stack([p.scale for p in parts]), "tile")

    gate, up, down = quantised(inner, hidden), quantised(inner, hidden), quantised(hidden, inner)
    router = (torch.randn(count, hidden, device="cuda") * hidden ** -0.5).bfloat16()
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    out, ids, gates = g.moe_fp8(x, router, gate, up, down, top_k)
    alone = torch.cat([g.moe_fp8(x[i:i + 1], router, gate, up, down, top_k)[0]
                       for i in range(tokens)])
    off = float((alone.float() - out.float()).norm() / out.float().norm())
    return out, ids, gates, off


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    g = Gemm(torch.device("cuda", 0))
    torch.manual_seed(0)
    losses, w, target = train(g, a.hidden, a.steps)
    print("training: mean square error %.4f -> %.4f in %d steps" % (losses[0], losses[-1], a.steps))
    off = serve(g, w, target)
    print("serving single rows: relative error against the target map %.3f" % off)
    out, ids, gates, drift = experts(g, a.hidden, a.hidden // 2)
    print("expert layer: %d tokens, experts of token 0: %s; one by one against together: %.1e"
          % (out.shape[0], ids[0].tolist(), drift))
    g.status()
    g.close()
    return losses, off, drift


if __name__ == "__main__":
    main()
