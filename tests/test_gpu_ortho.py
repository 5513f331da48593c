"""Orthogonalising on the GPU against its formula in doubles, and against a simulation in
doubles of what it rounds."""
import ctypes

import numpy as np
import pytest
import torch

from dense_gemm_tmem_gb300 import binding as B
from dense_gemm_tmem_gb300.gemm import Gemm

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
FAST, CONVERGENT = (3.4445, -4.7750, 2.0315), (1.875, -1.25, 0.375)


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    h = Gemm(torch.device("cuda", 0))
    yield h
    h.close()


def steps_of(abc, steps):
    return [abc] * steps if not hasattr(abc[0], "__len__") else list(abc)


def simulate(G, steps, abc, eps=1e-7, round16=True):
    """The steps in doubles; with round16, X, A and bA + cA² are rounded to fp16 where the
    products read them (relative to their magnitude, which is what scaling by powers of two
    makes of it), the iterate to fp32."""
    X = G.double()
    X = X / max(float(torch.linalg.matrix_norm(X)), eps)
    tall = X.shape[0] > X.shape[1]
    X = X.mT.contiguous() if tall else X
    r = (lambda v: (v * 4096).half().double() / 4096) if round16 else (lambda v: v)
    for a, b, c in steps_of(abc, steps):
        H = r(X)
        A = r(H @ H.mT)
        X = a * X + r(b * A + c * (A @ A)) @ H
        if round16:
            X = X.float().double()
    return X.mT if tall else X


def rel(a, b):
    return float((a - b).norm() / b.norm()) if float(b.norm()) else float(a.norm())


def check(got, G, steps, abc, eps=1e-7):
    """fp32 sums in another order turn over a few of the fp16 roundings, each by one step
    (2^-11 of an element): less than the roundings themselves, and the result's own rounding
    to bfloat16 is at most 2^-9 in the mean square (2^-8 at worst for an element)."""
    assert got.dtype == BF16 and got.shape == G.shape
    exact = simulate(G, steps, abc, eps, False)
    rounded = simulate(G, steps, abc, eps)
    own = rel(rounded, exact)
    assert rel(got.double(), exact) <= 1.5 * own + 2.0 ** -9 + 1e-6, (own, rel(got.double(), exact))


def gradient(rows, cols, dtype, rank=8, noise=0.05):
    rank = min(rank, rows, cols)
    fall = 1.0 / torch.arange(1, rank + 1, device="cuda")
    G = (torch.randn(rows, rank, device="cuda") * fall) @ torch.randn(rank, cols, device="cuda")
    return ((G + noise * torch.randn(rows, cols, device="cuda")) * 1e-3).to(dtype)


SHAPES = [(1, 1), (1, 64), (64, 1), (8, 8), (7, 33), (130, 67), (64, 257), (257, 64), (128, 128),
          (200, 300), (384, 640), (512, 512), (515, 1000), (1000, 515), (129, 2056), (700, 1000)]


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_shapes(g, rows, cols):
    torch.manual_seed(rows * 3 + cols)
    for dtype in (F32, BF16, F16):
        for G in (gradient(rows, cols, dtype), torch.randn(rows, cols, device="cuda").to(dtype)):
            check(g.orthogonalize(G), G, 5, FAST)
    g.status()


@pytest.mark.parametrize("rows,cols", [(100, 300), (600, 260), (1024, 1024)])
@pytest.mark.parametrize("abc,steps", [(FAST, 1), (FAST, 2), (CONVERGENT, 12), ((1.5, -0.5, 0.0), 9),
                                       ((1.0, 0.0, 0.0), 2), ((0.0, 1.0, 0.0), 1),
                                       ([(4.0, -6.0, 3.0), FAST, CONVERGENT], 3)])
def test_coefficients(g, rows, cols, abc, steps):
    torch.manual_seed(steps)
    G = torch.randn(rows, cols, device="cuda")
    check(g.orthogonalize(G, steps, abc), G, steps, abc)


def test_coefficients_changed_in_place(g):
    """A schedule held in tensors and changed between two calls."""
    torch.manual_seed(12)
    G = torch.randn(70, 130, device="cuda")
    for abc in (torch.tensor([FAST] * 3), tuple(torch.tensor(FAST) for _ in range(3))):
        assert torch.equal(g.orthogonalize(G, 3, abc), g.orthogonalize(G, 3, FAST))
        for row in abc:
            row.copy_(torch.tensor(CONVERGENT))
        assert torch.equal(g.orthogonalize(G, 3, abc), g.orthogonalize(G, 3, CONVERGENT))


def test_converges_to_the_polar_factor(g):
    torch.manual_seed(1)
    for rows, cols in ((96, 200), (300, 128)):
        q = torch.linalg.qr(torch.randn(max(rows, cols), min(rows, cols), device="cuda").double())[0]
        u = torch.linalg.qr(torch.randn(min(rows, cols), min(rows, cols), device="cuda").double())[0]
        s = torch.linspace(0.2, 1.0, min(rows, cols), device="cuda").double()
        P = q @ (u * s) @ u.T
        want, G = q, P
        if rows < cols:
            want, G = want.mT, G.mT
        got = g.orthogonalize(G.float().contiguous(), 16, CONVERGENT).double()
        # 16-bit operands in the last steps (2^-11 each) and the result's rounding
        assert rel(got, want.contiguous()) <= 3 * 2.0 ** -11 + 2.0 ** -9


@pytest.mark.parametrize("batch,rows,cols", [(1, 64, 100), (3, 70, 130), (10, 200, 72), (40, 128, 128),
                                             (5, 300, 260)])
def test_batch_is_each_by_itself(g, batch, rows, cols):
    torch.manual_seed(batch)
    G = torch.randn(batch, rows, cols, device="cuda") * torch.logspace(-6, 6, batch,
                                                                      device="cuda").view(-1, 1, 1)
    got = g.orthogonalize(G)
    for i in range(batch):
        check(got[i], G[i], 5, FAST)
        assert torch.equal(got[i], g.orthogonalize(G[i].contiguous())), i


def test_strided_input(g):
    torch.manual_seed(5)
    buf = torch.randn(4, 150, 260, device="cuda")
    for G in (buf[1:3, 3:130, 1:200], buf[::2, :100, :256], buf[0, ::3, 5:71],
              buf[:1].expand(3, 150, 260)):
        got = g.orthogonalize(G)
        assert got.is_contiguous() and torch.equal(got, g.orthogonalize(G.contiguous()))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e12, 3e37])
def test_far_magnitudes(g, dtype, scale):
    """Squares that leave fp32's range; eps far below."""
    torch.manual_seed(2)
    G = (torch.randn(130, 200, device="cuda").clamp(-5, 5).double() * scale).to(dtype)
    check(g.orthogonalize(G, eps=2.0 ** -100), G, 5, FAST, 2.0 ** -100)
    G[3, 4] = 3e38
    check(g.orthogonalize(G, eps=2.0 ** -100), G, 5, FAST, 2.0 ** -100)


def test_zero_small_and_non_finite(g):
    z = torch.zeros(3, 100, 64, device="cuda")
    assert float(g.orthogonalize(z).abs().max()) == 0
    z[1] = torch.randn(100, 64, device="cuda") * 1e-9
    got = g.orthogonalize(z)
    check(got[1], z[1], 5, FAST)
    assert float(got[0].abs().max()) == 0 and float(got[2].abs().max()) == 0
    for bad in (float("nan"), float("inf")):
        z[2, 99, 63] = bad
        again = g.orthogonalize(z)
        assert torch.equal(again[:2], got[:2]) and bool(torch.isnan(again[2]).all())


def test_empty(g):
    for shape in ((0, 5), (5, 0), (0, 4, 4), (3, 0, 4)):
        assert g.orthogonalize(torch.zeros(shape, device="cuda")).shape == shape


def test_streams_graphs_and_repeats(g):
    torch.manual_seed(3)
    for shape in ((64, 64), (3, 200, 136), (600, 1030)):
        G = torch.randn(shape, device="cuda").bfloat16()
        want = g.orthogonalize(G)
        for _ in range(4):
            assert torch.equal(g.orthogonalize(G), want)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = g.orthogonalize(G, stream=s)
        s.synchronize()
        assert torch.equal(got, want)
        graph, static = torch.cuda.CUDAGraph(), torch.randn_like(G)
        with torch.cuda.graph(graph):
            out = g.orthogonalize(static)
        static.copy_(G)
        for _ in range(3):
            graph.replay()
            assert torch.equal(out, want)
    g.status()


def run_c(g, p, abc, poison):
    """The C entry with a workspace of one byte's value throughout."""
    c = (ctypes.c_float * (3 * p.steps))(*(abc * p.steps))
    p.coefficients = ctypes.addressof(c)
    rc, size = B.gemm_orthogonalize_workspace(g.handle, p)
    assert rc == 0
    ws = torch.full((size,), poison, dtype=torch.uint8, device="cuda")
    rc = B.gemm_orthogonalize(g.handle, p, ws.data_ptr(), size,
                              torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    g.status()


@pytest.mark.parametrize("pair,tile_n", [(-1, -1), (0, -1), (1, 128), (1, 256)])
@pytest.mark.parametrize("batch,rows,cols", [(1, 1, 1), (1, 200, 131), (3, 70, 130), (2, 300, 261)])
def test_in_place_padded_and_any_workspace(g, pair, tile_n, batch, rows, cols):
    """out in rows and matrices with gaps, which stay as they were, or over g itself; the
    workspace's contents do not matter."""
    torch.manual_seed(cols)
    G = torch.randn(batch, rows, cols, device="cuda").bfloat16()
    g.set_option(B.GEMM_OPT_PAIR, pair)
    g.set_option(B.GEMM_OPT_FORCE_TILE_N, tile_n)
    try:
        want = g.orthogonalize(G)
        for pad, gap, place, poison in ((0, 0, False, 0xff), (5, 7, False, 0x7c), (3, 16, True, 0xff),
                                        (8, 64, True, 0)):
            ld = cols + pad
            stride = rows * ld + gap
            buf = torch.full((batch * stride + 8,), 7.0, device="cuda").bfloat16()
            view = buf.as_strided((batch, rows, cols), (stride, ld, 1), 1)
            src = G
            if place:
                view.copy_(G)
                src = view
            p = B.gemm_orthogonalize_t(batch=batch, rows=rows, cols=cols, steps=5, dtype=B.GEMM_BF16,
                                       eps=1e-7, g=src.data_ptr(), ld_g=src.stride(1),
                                       stride_g=src.stride(0), out=view.data_ptr(), ld_out=ld,
                                       stride_out=stride)
            run_c(g, p, FAST, poison)
            assert torch.equal(view, want)
            view.fill_(7.0)
            assert bool((buf == 7.0).all())
    finally:
        g.set_option(B.GEMM_OPT_PAIR, -1)
        g.set_option(B.GEMM_OPT_FORCE_TILE_N, -1)


@pytest.mark.parametrize("abc", [[(2.0 ** -20, 0.0, 0.0), (2.0 ** 20, 0.0, 0.0), FAST],
                                 [(2.0 ** -10, 0.0, 0.0), (0.0, 2.0 ** 30, 0.0), FAST],
                                 [(0.01, 0.0, 0.0), (150.0, -8e5, 1e9), FAST],
                                 [(1.0, 0.0, 0.0), (2.0 ** -40, 2.0 ** -40, 0.0)]])
def test_an_iterate_far_below_1(g, abc):
    """The 16-bit copies' scales follow it.  (The result itself may be far below 1: relative.)"""
    torch.manual_seed(6)
    for rows, cols in ((40, 100), (130, 64)):
        G = torch.randn(rows, cols, device="cuda")
        got = g.orthogonalize(G, len(abc), abc)
        exact = simulate(G, len(abc), abc, round16=False)
        # each copy's 2^-11, up to four of them in a step's product, three steps, whose
        # coefficients magnify by less than 4; the result's rounding
        assert rel(got.double(), exact) <= 12 * 4 * 2.0 ** -11 + 2.0 ** -9
    g.status()


def test_two_graphs_at_once(g):
    """Each has scratch of its own."""
    torch.manual_seed(8)
    G = [torch.randn(300, 520, device="cuda"), torch.randn(2, 260, 200, device="cuda")]
    want = [g.orthogonalize(x) for x in G]
    graphs, outs = [], []
    for x in G:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(g.orthogonalize(x))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in G]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    g.status()


@pytest.mark.parametrize("pair,tile_n", [(0, -1), (1, 128), (1, 256)])
@pytest.mark.parametrize("batch,rows,cols", [(1, 130, 70), (2, 300, 600), (3, 600, 270),
                                             (1, 700, 700), (5, 64, 40)])
def test_every_tile_on_every_shape(g, pair, tile_n, batch, rows, cols):
    """One CTA's tiles, and both of a pair's, whatever the rule would take."""
    torch.manual_seed(rows)
    G = torch.randn(batch, rows, cols, device="cuda")
    g.set_option(B.GEMM_OPT_PAIR, pair)
    g.set_option(B.GEMM_OPT_FORCE_TILE_N, tile_n)
    try:
        for steps, abc in ((5, FAST), (2, CONVERGENT)):
            got = g.orthogonalize(G, steps, abc)
            for i in range(batch):
                check(got[i], G[i], steps, abc)
            assert torch.equal(g.orthogonalize(G, steps, abc), got)
        g.status()
    finally:
        g.set_option(B.GEMM_OPT_PAIR, -1)
        g.set_option(B.GEMM_OPT_FORCE_TILE_N, -1)


@pytest.mark.parametrize("pair,tile_n", [(0, -1), (1, 128), (1, 256)])
def test_under_short_wait_limits(g, pair, tile_n):
    """Limits that run out anywhere in the launch: it ends, gemm_status reports it or the
    result is right, and the next call is right."""
    from test_gpu_fp8_limits import limited
    torch.manual_seed(4)
    G = torch.randn(2, 520, 600, device="cuda")
    g.set_option(B.GEMM_OPT_PAIR, pair)
    g.set_option(B.GEMM_OPT_FORCE_TILE_N, tile_n)
    try:
        limited(g, lambda: [g.orthogonalize(G)], [1, 300, 1000, 3000, 10000, 30000], times=3)
    finally:
        g.set_option(B.GEMM_OPT_PAIR, -1)
        g.set_option(B.GEMM_OPT_FORCE_TILE_N, -1)


def check_elements(got, G, steps, abc):
    """Every element by itself.  Its error is a sum of hundreds of roundings to fp16, as the
    simulation's is, whose rms over the element's row or column (the larger) is s; the two
    need not round alike, but a sum of independent bounded roundings is beyond 10 s once in
    e^50 (Hoeffding).  Truncating fp32 sums of 5000 products lose 2^-23 of themselves for each
    16, a tenth of what 2^-12 of each operand makes of them.  The result's rounding to bfloat16
    comes on top, half a step, 2^-8.  An element that is missing or another's is off by its
    own size: some 500 s."""
    exact = simulate(G, steps, abc, round16=False)
    e = (simulate(G, steps, abc) - exact).square()
    s = torch.maximum(e.mean(1, keepdim=True).sqrt(), e.mean(0, keepdim=True).sqrt())
    tol = 2.0 ** -8 * exact.abs() + 10 * (1 + 2.0 ** -8) * s
    off = (got.double() - exact).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist(), float((off / tol).max()))


@pytest.mark.parametrize("pair,tile_n", [(-1, -1), (0, -1), (1, 128), (1, 256)])
@pytest.mark.parametrize("batch,rows,cols", [(1, 130, 70), (1, 64, 257), (1, 257, 64), (2, 300, 600),
                                             (3, 600, 270), (1, 515, 1000), (1, 1000, 515),
                                             (2, 700, 1000), (1, 129, 2056), (1, 40, 5000)])
def test_every_element_on_every_tile(g, pair, tile_n, batch, rows, cols):
    """Tile corners, ragged ends and mirrored blocks, of which a matrix's norm says little."""
    torch.manual_seed(rows + 2 * cols)
    G = torch.randn(batch, rows, cols, device="cuda")
    G[-1] = gradient(rows, cols, F32)
    g.set_option(B.GEMM_OPT_PAIR, pair)
    g.set_option(B.GEMM_OPT_FORCE_TILE_N, tile_n)
    try:
        for steps, abc in ((5, FAST), (3, CONVERGENT)):
            got = g.orthogonalize(G, steps, abc)
            for i in range(batch):
                check_elements(got[i], G[i], steps, abc)
        g.status()
    finally:
        g.set_option(B.GEMM_OPT_PAIR, -1)
        g.set_option(B.GEMM_OPT_FORCE_TILE_N, -1)
