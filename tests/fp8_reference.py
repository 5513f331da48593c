"""64-bit reference of the block-scaled 8-bit operators, on the host, and the
error bounds their fp32 arithmetic allows."""
from __future__ import annotations

import numpy as np
import torch

BLOCK = 128
SHAPE = {"row": (1, BLOCK), "col": (BLOCK, 1), "tile": (BLOCK, BLOCK)}
AMAX_MIN = 2.0 ** -100
U32 = 2.0 ** -24                                 # half an ulp of fp32, relative
OUT_U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
OUT_TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}


def round_e4m3(v):
    """Doubles to the nearest e4m3 value, ties to even (NaN stays NaN)."""
    v = np.asarray(v, np.float64)
    a = np.abs(np.where(np.isfinite(v), v, 0.0))
    _, e = np.frexp(a)
    step = np.exp2(np.maximum(e - 1, -6) - 3)
    q = np.sign(np.where(np.isnan(v), 0.0, v)) * np.minimum(np.round(a / step) * step, 448.0)
    return np.where(np.isfinite(v), q, np.nan)


def spread(s, rows, cols, blocks):
    br, bc = SHAPE[blocks]
    return np.repeat(np.repeat(s, br, -2)[..., :rows, :], bc, -1)[..., :cols]


def quantize(x, blocks):
    """(values, scales): the definition, with the fp32 roundings it names."""
    x = np.asarray(x, np.float64)
    R, C = x.shape
    br, bc = SHAPE[blocks]
    rb, cb = -(-R // br), -(-C // bc)
    a = np.zeros((rb * br, cb * bc))
    a[:R, :C] = np.where(np.isfinite(x), np.abs(x), 0.0)
    amax = np.maximum(a.reshape(rb, br, cb, bc).max((1, 3)), AMAX_MIN)
    scale = (amax / 448.0).astype(np.float32)
    inv = (448.0 / amax).astype(np.float32).astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        p = (x * spread(inv, R, C, blocks)).astype(np.float32).astype(np.float64)
    return round_e4m3(p), scale


def values(q, s, blocks):
    q = np.asarray(q, np.float64)
    return q * spread(np.asarray(s, np.float64), *q.shape[-2:], blocks)


def host(t):
    """A tensor's values as doubles."""
    if t.dtype in (torch.float8_e4m3fn, torch.uint8):
        t = t.view(torch.float8_e4m3fn).float()
    return t.detach().double().cpu().numpy()


def product_bound(a, b, want, out_dtype):
    """Largest error an fp32-accumulated product may have: in a k-block at most
    128 additions, each off by at most an ulp of a partial sum (the tensor cores
    truncate), then one fused add a k-block, the scales' product and their
    conversion; all relative to sum |a b|.  Plus one rounding to the output type."""
    K = a.shape[1]
    steps = min(K, BLOCK) + -(-K // BLOCK) + 4
    mag = np.abs(a) @ np.abs(b)
    err = 2 * U32 * steps * mag
    return err + OUT_U[out_dtype] * (np.abs(want) + err) + OUT_TINY[out_dtype]


def check_choice(x, router, ids):
    """Whether ids (T, k) are the experts of the largest logits in descending
    order, as far as fp32 logits (H additions each) can tell: k different ones,
    each of a logit within the error of the one that belongs there."""
    T, H = x.shape
    logits = x @ router.T
    e_log = (H + 2) * U32 * (np.abs(x) @ np.abs(router).T)
    top = -np.sort(-logits, axis=1)[:, :ids.shape[1]]
    got = np.take_along_axis(logits, ids, 1)
    assert all(len(set(r)) == len(r) for r in ids.tolist())
    assert (np.abs(got - top) <= 2 * e_log.max(1, keepdims=True)).all()


def moe(x, router, w1, w3, w2, ids, renorm):
    """The layer in doubles for the chosen experts, and a bound on each output's
    error.  x (T, H), router (E, H), w1, w3 (E, I, H), w2 (E, H, I): stored
    values as doubles; ids (T, k)."""
    T, H = x.shape
    E, I, _ = w1.shape
    top_k = ids.shape[1]
    logits = x @ router.T
    # logits: H additions in fp32
    e_log = (H + 2) * U32 * (np.abs(x) @ np.abs(router).T)
    p = np.exp(logits - logits.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    g = np.take_along_axis(p, ids, 1)
    if renorm:
        g = g / g.sum(1, keepdims=True)
    # a gate's relative error: twice the logits' (numerator and sum), and the
    # fp32 exp, sum and division (E additions)
    e_g = (2 * 2 * e_log.max(1, keepdims=True) + (E + 16) * U32) * g
    q, s = quantize(x, "row")
    xq = values(q, s, "row")
    out, slack = np.zeros((T, H)), np.zeros((T, H))
    kh, ki = min(H, BLOCK) + -(-H // BLOCK) + 4, min(I, BLOCK) + -(-I // BLOCK) + 4
    for t in range(T):
        for j in range(top_k):
            e = ids[t, j]
            a, b = w1[e] @ xq[t], w3[e] @ xq[t]
            ea = 2 * U32 * kh * (np.abs(w1[e]) @ np.abs(xq[t]))
            eb = 2 * U32 * kh * (np.abs(w3[e]) @ np.abs(xq[t]))
            silu = a / (1 + np.exp(-a))
            h = silu * b
            # |silu'| <= 1.1; exp, division and two products in fp32
            eh = np.abs(silu) * eb + 1.1 * np.abs(b) * ea + 16 * U32 * np.abs(h) + ea * eb
            hq, hs = quantize(h[None], "row")
            hv = values(hq, hs, "row")[0]
            # what rounding to e4m3 can turn an error of eh, and of the block's maximum, into
            inv = 1.0 / spread(hs.astype(np.float64), 1, I, "row")[0]
            amax = spread(hs.astype(np.float64), 1, I, "row")[0] * 448
            ehb = np.array([eh[k // BLOCK * BLOCK:(k // BLOCK + 1) * BLOCK].max()
                            for k in range(0, I, BLOCK)])
            rel = np.repeat(ehb, BLOCK)[:I] / amax + 4 * U32
            d = eh + np.abs(h) * rel
            lo, hi = round_e4m3((h - d) * inv), round_e4m3((h + d) * inv)
            ev = (hi - lo) / inv + np.abs(hv) * rel
            y = w2[e] @ hv
            ey = np.abs(w2[e]) @ ev + 2 * U32 * ki * (np.abs(w2[e]) @ (np.abs(hv) + ev))
            out[t] += g[t, j] * y
            slack[t] += g[t, j] * ey + e_g[t, j] * (np.abs(y) + ey) + 4 * U32 * np.abs(g[t, j] * y)
        slack[t] += top_k * U32 * np.abs(out[t])
    return out, slack, g, e_g
