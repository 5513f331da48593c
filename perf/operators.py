"""The block-scaled 8-bit operators: cases, inputs, a plain form and a 64-bit definition of each.

Four operators that run together in a linear layer trained, and a mixture-of-experts layer served,
in 8-bit floating point (e4m3) with one fp32 scale for each block of 128:

  quantize   a matrix to e4m3 with scales of 1 x 128 ("row"), 128 x 1 ("col"), both at once
             ("row+col") or 128 x 128 ("tile") blocks
  product    C = A.B (+bias) of two such matrices, every storage order, fp32 accumulation
  linear     one training step of a linear layer on them: y, dx and dW from x, W and dy
  moe        a whole mixture-of-experts layer for a few tokens: router, top-k, gate/up/down products
             of the chosen experts with 8-bit weights, weighted sum

A quantised block holds s = max(amax, 2^-100) / 448 and q = e4m3(x * (448 / max(amax, 2^-100))), with
amax over the block's finite elements; non-finite elements are stored as NaN.

`own` selects the framework's kernels (True) or elementary torch operations in fp32 (False).
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -100
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------- cases --
def listed():
    return [
        # one token's activations before a decode product: latency only
        dict(name="quant_row_1x4096_f16", op="quantize", rows=1, cols=4096, dtype="f16",
             blocks="row"),
        # a training step's activations, quantised along both axes in one pass
        dict(name="quant_both_8192x8192_bf16", op="quantize", rows=8192, cols=8192, dtype="bf16",
             blocks="row+col"),
        # fp32 master weights of a ragged layer, before each step
        dict(name="quant_tile_2050x5000_f32", op="quantize", rows=2050, cols=5000, dtype="f32",
             blocks="tile"),
        # decode of one token, and of a batch of 64, through one 4096 x 4096 weight
        dict(name="prod_1x4096x4096_f16", op="product", M=1, N=4096, K=4096, a_major="row",
             b_major="col", b_blocks="tile", out="f16", bias=False),
        dict(name="prod_64x4096x4096_bf16", op="product", M=64, N=4096, K=4096, a_major="row",
             b_major="col", b_blocks="tile", out="bf16", bias=False),
        # a ragged prompt, odd depth, with a bias
        dict(name="prod_1001x2050x4100_f16_bias", op="product", M=1001, N=2050, K=4100,
             a_major="row", b_major="col", b_blocks="tile", out="f16", bias=True),
        # the benchmark's square size
        dict(name="prod_8192x8192x8192_f16", op="product", M=8192, N=8192, K=8192, a_major="row",
             b_major="col", b_blocks="tile", out="f16", bias=False),
        # one training step of a layer: forward, input gradient, weight gradient
        dict(name="linear_4096x4096x4096_bf16", op="linear", T=4096, N=4096, K=4096, dtype="bf16"),
        dict(name="linear_515x1000x2056_f16", op="linear", T=515, N=1000, K=2056, dtype="f16"),
        # decode of one token through 8 of 64 experts
        dict(name="moe_1x2048x1024_e64k8_bf16", op="moe", T=1, H=2048, I=1024, E=64, k=8,
             dtype="bf16", renorm=True),
        # a ragged layer, a handful of tokens
        dict(name="moe_5x1000x700_e10k3_f16", op="moe", T=5, H=1000, I=700, E=10, k=3,
             dtype="f16", renorm=False),
        # a decode batch that touches most of 128 experts
        dict(name="moe_32x4096x1024_e128k8_bf16", op="moe", T=32, H=4096, I=1024, E=128, k=8,
             dtype="bf16", renorm=True),
    ]


def _log(rng, lo, hi):
    """A size between lo and hi, even over the logarithm: two in three as they fall, one in three
    rounded down to a multiple of 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 1 / 3 and v >= 64:
        v = v // 64 * 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "linear", "moe", "moe"])
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 8192),
                    dtype=rng.choice(sorted(TYPES)),
                    blocks=rng.choice(["row", "col", "row+col", "tile"]))
    if op == "product":
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 64, 8192), K=_log(rng, 64, 8192),
                    a_major=rng.choice(["row", "row", "col"]),
                    b_major=rng.choice(["col", "row"]), b_blocks=rng.choice(["tile", "line"]),
                    out=rng.choice(sorted(TYPES)), bias=rng.random() < 0.3)
    if op == "linear":
        return dict(op=op, T=_log(rng, 128, 4096), N=_log(rng, 256, 4096), K=_log(rng, 256, 4096),
                    dtype=rng.choice(["f16", "bf16"]))
    E = rng.choice([8, 10, 16, 32, 60, 64, 128])
    return dict(op=op, T=_log(rng, 1, 32), H=_log(rng, 512, 4096), I=_log(rng, 256, 1024), E=E,
                k=rng.choice([1, 2, 4, 6, 8]), dtype=rng.choice(["f16", "bf16"]),
                renorm=rng.random() < 0.5)


def _ceil(a, b):
    return -(-a // b)


def _scales(rows, cols, kind):
    """How many scales a rows x cols matrix has."""
    return {"row": rows * _ceil(cols, BLOCK), "col": _ceil(rows, BLOCK) * cols,
            "tile": _ceil(rows, BLOCK) * _ceil(cols, BLOCK)}[kind]


def work(case):
    c = case
    size = {"f16": 2, "bf16": 2, "f32": 4}
    if c["op"] == "quantize":
        n = c["rows"] * c["cols"]
        kinds = c["blocks"].split("+")
        return {"bytes": n * size[c["dtype"]] + sum(n + 4 * _scales(c["rows"], c["cols"], k)
                                                    for k in kinds), "flops": 2 * n * len(kinds)}
    if c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        sb = _scales(N, K, "row" if c["b_blocks"] == "line" else "tile")
        return {"bytes": M * K + N * K + 4 * (_scales(M, K, "row") + sb) + M * N * size[c["out"]]
                + (4 * N if c["bias"] else 0), "flops": 2 * M * N * K}
    if c["op"] == "linear":
        T, N, K, s = c["T"], c["N"], c["K"], size[c["dtype"]]
        # x, W, dy read; y, dx, dW (fp32) written
        return {"bytes": s * (T * K + N * K + T * N) + s * (T * N + T * K) + 4 * N * K,
                "flops": 6 * T * N * K}
    T, H, I, E, k, s = c["T"], c["H"], c["I"], c["E"], min(c["k"], c["E"]), size[c["dtype"]]
    chosen = E * (1 - (1 - k / E) ** T)  # experts that some token chose, if all are as likely
    weights = 3 * H * I + 4 * 3 * _ceil(H, BLOCK) * _ceil(I, BLOCK)
    return {"bytes": chosen * weights + s * (E * H + 2 * T * H) + 8 * T * k,
            "flops": 2 * T * k * 3 * H * I + 2 * T * E * H}


# --------------------------------------------------------------- plain operators --
def _blocks_amax(x, br, bc):
    """max |x| over the finite elements of each br x bc block of a 2-D fp32 matrix."""
    R, C = x.shape
    a = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    a = torch.nn.functional.pad(a, (0, _ceil(C, bc) * bc - C, 0, _ceil(R, br) * br - R))
    return a.view(_ceil(R, br), br, _ceil(C, bc), bc).amax(dim=(1, 3))


def _spread(s, R, C, br, bc):
    """The scale of each element."""
    return s.repeat_interleave(br, 0)[:R].repeat_interleave(bc, 1)[:, :C]


_SHAPE = {"row": (1, BLOCK), "col": (BLOCK, 1), "tile": (BLOCK, BLOCK)}


def _quantize(x, kind):
    br, bc = _SHAPE[kind]
    x = x.float()
    amax = _blocks_amax(x, br, bc).clamp_min(AMAX_MIN)
    inv = torch.full_like(amax, E4M3_MAX) / amax
    q = (x * _spread(inv, *x.shape, br, bc)).to(torch.float8_e4m3fn)
    # a true division: torch multiplies by the reciprocal where the divisor is a Python number
    return q, amax / torch.full_like(amax, E4M3_MAX)


def _dequantize(q, s, kind):
    br, bc = _SHAPE[kind]
    return q.float() * _spread(s, *q.shape, br, bc)


def _plain_moe(st):
    c, x = st["case"], st["x"].float()
    T, H, k = c["T"], c["H"], min(c["k"], c["E"])
    logits = x @ st["router"].float().t()
    prob = torch.softmax(logits, 1)
    ids = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k]
    gates = prob.gather(1, ids)
    if c["renorm"]:
        gates = gates / gates.sum(1, keepdim=True)
    xq = _dequantize(*_quantize(x, "row"), "row")

    def experts(w, s, v):  # the chosen experts' rows, one product for each choice
        w = w[ids.reshape(-1)].float()
        P, R, C = w.shape
        s = s[ids.reshape(-1)].repeat_interleave(BLOCK, 1)[:, :R]
        w *= s.repeat_interleave(BLOCK, 2)[:, :, :C]
        return torch.bmm(w, v.unsqueeze(2)).squeeze(2)

    v = xq.repeat_interleave(k, 0)
    g, u = experts(*st["w1"], v), experts(*st["w3"], v)
    h = g * torch.sigmoid(g) * u
    h = _dequantize(*_quantize(h, "row"), "row")
    y = experts(*st["w2"], h).view(T, k, H)
    return {"out": (y * gates.unsqueeze(2)).sum(1).to(st["x"].dtype), "ids": ids.int(),
            "gates": gates}


# ----------------------------------------------------------------------- inputs --
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _activations(g, rows, cols):
    """Normal values with a few channels an order of magnitude larger."""
    x = _normal(g, rows, cols)
    hot = torch.rand(cols, generator=g, device="cuda") < 0.005
    return torch.where(hot, 12.0 * x, x)


def _padded(q):
    """The same values with rows 16-byte aligned, as the framework's quantiser lays them."""
    *lead, cols = q.shape
    buf = torch.zeros(*lead, _ceil(cols, 16) * 16, dtype=q.dtype, device=q.device)
    buf[..., :cols] = q
    return buf[..., :cols]


def _laid(q, s, kind):
    """Quantised storage as the framework's quantiser writes it: padded rows, and for 1 x 128
    blocks the scales of one k-block next to each other."""
    return _padded(q), (s.t().contiguous().t() if kind == "row" else s.contiguous())


def prepare(case, seed):
    c = dict(case)
    g = _gen(seed)
    st = {"case": c}
    if c["op"] == "quantize":
        st["x"] = _activations(g, c["rows"], c["cols"]).to(TYPES[c["dtype"]])
    elif c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        a, b = _activations(g, M, K), _normal(g, N, K) * K ** -0.5
        # A is stored M x K or K x M, B N x K ("col") or K x N ("row"); the blocks run along K
        ka = "row" if c["a_major"] == "row" else "col"
        kb = "tile" if c["b_blocks"] == "tile" else "row" if c["b_major"] == "col" else "col"
        a = a if c["a_major"] == "row" else a.t()
        b = b if c["b_major"] == "col" else b.t()
        st["A"], st["B"] = _laid(*_quantize(a, ka), ka), _laid(*_quantize(b, kb), kb)
        st["kinds"] = (ka, kb)
        st["bias"] = _normal(g, N) if c["bias"] else None
    elif c["op"] == "linear":
        t = TYPES[c["dtype"]]
        st["x"] = _activations(g, c["T"], c["K"]).to(t)
        st["w"] = (_normal(g, c["N"], c["K"]) * c["K"] ** -0.5).to(t)
        st["dy"] = (_normal(g, c["T"], c["N"]) * 1e-3).to(t)
    else:
        T, H, I, E, t = c["T"], c["H"], c["I"], c["E"], TYPES[c["dtype"]]
        st["x"] = _normal(g, T, H).to(t)
        st["router"] = (_normal(g, E, H) * H ** -0.5).to(t)

        def weights(rows, cols):
            q = _normal(g, E, rows, cols, dtype=torch.float16).mul_(112).clamp_(-448, 448)
            s = (0.5 + torch.rand(E, _ceil(rows, BLOCK), _ceil(cols, BLOCK), generator=g,
                                  device="cuda")) / (112 * cols ** 0.5)
            return _padded(q.to(torch.float8_e4m3fn)), s

        st["w1"], st["w3"], st["w2"] = weights(I, H), weights(I, H), weights(H, I)
    return st


# -------------------------------------------------------------------------- run --
_handle = None


def _gemm():
    """The program's one library handle."""
    global _handle
    if _handle is None:
        from dense_gemm_tmem_gb300.gemm import Gemm
        _handle = Gemm(torch.device("cuda", torch.cuda.current_device()))
    return _handle


def _run_own(st):
    from dense_gemm_tmem_gb300 import fp8
    c, g = st["case"], _gemm()
    if c["op"] == "quantize":
        r = g.fp8_quantize(st["x"], c["blocks"])
        if c["blocks"] == "row+col":
            return {"row": [r[0].data, r[0].scale], "col": [r[1].data, r[1].scale]}
        return {c["blocks"]: [r.data, r.scale]}
    if c["op"] == "product":
        if "B8" not in st:  # a program keeps its weight's object
            st["B8"] = fp8.Fp8Matrix(st["B"][0], st["B"][1], st["kinds"][1])
        A = fp8.Fp8Matrix(st["A"][0], st["A"][1], st["kinds"][0])
        return g.fp8_matmul(A, st["B8"], st["bias"], a_major=0 if c["a_major"] == "row" else 1,
                            b_major=0 if c["b_major"] == "row" else 1, out_dtype=TYPES[c["out"]])
    if c["op"] == "linear":
        y, saved = fp8.linear_forward(g, st["x"], st["w"])
        dx, dw = fp8.linear_backward(g, st["dy"], saved)
        return {"y": y, "dx": dx, "dw": dw}
    if "layer" not in st:
        st["layer"] = [fp8.Fp8Matrix(*st[w], "tile") for w in ("w1", "w3", "w2")]
    out, ids, gates = g.moe_fp8(st["x"], st["router"], *st["layer"], top_k=min(c["k"], c["E"]),
                                renormalize=c["renorm"])
    return {"out": out, "ids": ids, "gates": gates}


def run(state):
    if own:
        return _run_own(state)
    st, c = state, state["case"]
    if c["op"] == "quantize":
        return {k: list(_quantize(st["x"], k)) for k in c["blocks"].split("+")}
    if c["op"] == "product":
        a, b = _dequantize(*st["A"], st["kinds"][0]), _dequantize(*st["B"], st["kinds"][1])
        C = (a if c["a_major"] == "row" else a.t()) @ (b.t() if c["b_major"] == "col" else b)
        return (C + st["bias"] if c["bias"] else C).to(TYPES[c["out"]])
    if c["op"] == "linear":
        t = st["x"].dtype
        xr = _dequantize(*_quantize(st["x"], "row"), "row")
        xc = _dequantize(*_quantize(st["x"], "col"), "col")
        w = _dequantize(*_quantize(st["w"], "tile"), "tile")
        dr = _dequantize(*_quantize(st["dy"], "row"), "row")
        dc = _dequantize(*_quantize(st["dy"], "col"), "col")
        return {"y": (xr @ w.t()).to(t), "dx": (dr @ w).to(t), "dw": dc.t() @ xc}
    return _plain_moe(st)


# ------------------------------------------------------------------------ exact --
def _round_e4m3(v):
    """Doubles to the nearest e4m3 value, ties to even, as doubles (|v| <= 448)."""
    _, e = torch.frexp(v)  # |v| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 1, min=-6) - 3)
    return torch.round(v / step) * step


def _exact_quantize(x, kind):
    """(q, s, q * s) in doubles; every input here is finite.  x * 448 is exact and its quotient
    rounded once, so an element that lies on a tie between two e4m3 values is seen as one."""
    br, bc = _SHAPE[kind]
    x = x.double()
    R, C = x.shape
    pad = x.new_zeros(_ceil(R, br) * br, _ceil(C, bc) * bc)
    pad[:R, :C] = x
    tiles = pad.reshape(_ceil(R, br), br, _ceil(C, bc), bc)
    amax = tiles.abs().amax(3, keepdim=True).amax(1, keepdim=True).clamp_min(AMAX_MIN)
    s = amax / E4M3_MAX
    q = _round_e4m3(tiles * E4M3_MAX / amax)
    back = (q * s).reshape(pad.shape)[:R, :C]
    return q.reshape(pad.shape)[:R, :C], s.reshape(s.shape[0], s.shape[2]), back


def _exact_value(q, s):
    """Doubles of a stored matrix from its values and block scales (2-D)."""
    br, bc = _ceil(q.shape[0], s.shape[0]), _ceil(q.shape[1], s.shape[1])
    i = torch.arange(q.shape[0], device=q.device) // (1 if br == 1 else BLOCK)
    j = torch.arange(q.shape[1], device=q.device) // (1 if bc == 1 else BLOCK)
    return q.float().double() * s.double()[i][:, j]


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["op"] == "quantize":
        return {k: list(_exact_quantize(st["x"], k)[:2]) for k in c["blocks"].split("+")}
    if c["op"] == "product":
        a, b = _exact_value(*st["A"]), _exact_value(*st["B"])
        a = a.t() if c["a_major"] == "col" else a
        b = b.t() if c["b_major"] == "col" else b
        C = torch.mm(a, b)
        return C.add_(st["bias"].double()) if c["bias"] else C
    if c["op"] == "linear":
        w = _exact_quantize(st["w"], "tile")[2]
        y = torch.mm(_exact_quantize(st["x"], "row")[2], w.t())
        dx = torch.mm(_exact_quantize(st["dy"], "row")[2], w)
        dw = torch.mm(_exact_quantize(st["dy"], "col")[2].t(), _exact_quantize(st["x"], "col")[2])
        return {"y": y, "dx": dx, "dw": dw}
    k = min(c["k"], c["E"])
    x = st["x"].double()
    logits = torch.mm(x, st["router"].double().t())
    top, ids = torch.topk(logits, k, dim=1)
    norm = torch.logsumexp(top if c["renorm"] else logits, 1, keepdim=True)
    gates = torch.exp(top - norm)
    xq = _exact_quantize(st["x"], "row")[2]
    out = torch.zeros_like(x)
    for e in torch.unique(ids).tolist():
        t, j = torch.nonzero(ids == e, as_tuple=True)
        w1, w3, w2 = (_exact_value(st[w][0][e], st[w][1][e]) for w in ("w1", "w3", "w2"))
        gate, up = torch.mm(xq[t], w1.t()), torch.mm(xq[t], w3.t())
        h = _exact_quantize(gate / (1 + torch.exp(-gate)) * up, "row")[2]
        out.index_add_(0, t, gates[t, j].unsqueeze(1) * torch.mm(h, w2.t()))
    return {"out": out, "ids": None, "gates": gates}
