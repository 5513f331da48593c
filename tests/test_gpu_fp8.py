"""The block-scaled 8-bit operators on the GPU against a 64-bit reference:
quantising bit for bit, products and the expert layer within bounds derived
from their fp32 arithmetic, at the sizes, strides and values where they can go
wrong."""
import numpy as np
import pytest
import torch

import fp8_reference as R
from dense_gemm_tmem_gb300 import binding as B
from dense_gemm_tmem_gb300 import fp8
from dense_gemm_tmem_gb300.fp8 import Fp8Matrix
from dense_gemm_tmem_gb300.gemm import COL, ROW, Gemm

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    h = Gemm(torch.device("cuda", 0))
    yield h
    h.close()


def normal(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape))


def same_values(got, want):
    assert got.shape == want.shape
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.array_equal(got[ok], want[ok]), int((got[ok] != want[ok]).sum())


def check_quantized(m, x, blocks):
    q, s = R.quantize(R.host(x), blocks)
    same_values(R.host(m.data), q)
    assert np.array_equal(m.scale.cpu().numpy(), s)


# ------------------------------------------------------------------ quantise --
@pytest.mark.parametrize("blocks", ["row", "col", "row+col", "tile"])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 129), (128, 128), (127, 257),
                                       (260, 1000), (1, 4096), (700, 16)])
def test_quantize(g, rows, cols, dtype, blocks):
    rng = np.random.default_rng(rows * 1000 + cols)
    x = (normal(rng, rows, cols) * torch.exp(2 * normal(rng, 1, cols))).to(dtype).cuda()
    m = g.fp8_quantize(x, blocks)
    for part, kind in zip(m if isinstance(m, tuple) else (m,), blocks.split("+")):
        assert part.blocks == kind
        check_quantized(part, x, kind)


@pytest.mark.parametrize("blocks", ["row", "col", "row+col", "tile"])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_quantize_special_values(g, dtype, blocks):
    """Zero blocks, the smallest magnitudes, infinities and NaN: a non-finite
    element is NaN and leaves its block's scale alone."""
    rng = np.random.default_rng(7)
    x = normal(rng, 300, 300)
    x[0:128, 0:128] = 0.0
    x[130, :] = float("nan")
    x[140, 150] = float("inf")
    x[141, 5] = -float("inf")
    x[:, 290] = float("inf")
    x[200, 128:256] = torch.finfo(dtype).tiny
    x[201, 128:256] = torch.finfo(dtype).smallest_normal / 8
    x[202, 0:128] = torch.finfo(dtype).max
    x = x.to(dtype).cuda()
    m = g.fp8_quantize(x, blocks)
    for part, kind in zip(m if isinstance(m, tuple) else (m,), blocks.split("+")):
        check_quantized(part, x, kind)


@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 3), (8, 0), (3, 5)])
def test_quantize_strided_and_unaligned(g, offset, pad):
    rng = np.random.default_rng(offset + 10 * pad)
    rows, cols = 131, 300
    flat = normal(rng, rows * (cols + pad) + offset).half().cuda()
    x = torch.as_strided(flat, (rows, cols), (cols + pad, 1), offset)
    check_quantized(g.fp8_quantize(x, "row"), x, "row")
    a, b = g.fp8_quantize(x, "row+col")
    check_quantized(a, x, "row")
    check_quantized(b, x, "col")


def test_quantize_leaves_padding_alone(g):
    """Bytes between cols and ld are the caller's."""
    x = torch.ones(5, 21, dtype=F32, device="cuda")
    data = torch.full((5, 32), 0x5a, dtype=torch.uint8, device="cuda")
    m = Fp8Matrix(data[:, :21], torch.empty(5, 1, device="cuda"), "row")
    rc = B.gemm_fp8_quantize(g.handle, 5, 21, x.data_ptr(), 21, B.GEMM_F32, m.desc(), None,
                             torch.cuda.current_stream().cuda_stream)
    assert rc == B.GEMM_OK
    assert bool((data[:, 21:] == 0x5a).all()) and bool((data[:, :21] == 0x7e).all())


# ------------------------------------------------------------------- product --
def operand(g, rng, mn, K, k_rows, tile, pad=0, offset=0, row_scales=False):
    """A block-scaled operand (stored form and doubles as mn x K), with rows
    padded by `pad` bytes beyond 16-byte rows and the base moved by `offset`."""
    x = normal(rng, mn, K) * torch.exp(normal(rng, mn, 1))
    blocks = "tile" if tile else ("row" if k_rows else "col")
    x = (x if k_rows else x.t()).float().contiguous()
    r, c = x.shape
    q, s = R.quantize(x.numpy(), blocks)
    ld = -(-c // 16) * 16 + pad
    buf = torch.full((r * ld + offset + 16,), 0x7f, dtype=torch.uint8)  # NaN around the values
    view = torch.as_strided(buf, (r, c), (ld, 1), offset)
    view.copy_(torch.from_numpy(q).float().to(torch.float8_e4m3fn).view(torch.uint8))
    dev = buf.cuda()
    data = torch.as_strided(dev, (r, c), (ld, 1), offset)
    st = torch.from_numpy(s)
    scale = (st.t().contiguous().cuda().t() if not row_scales else st.cuda())
    v = R.values(q, s, blocks)
    return Fp8Matrix(data, scale, blocks), (v if k_rows else v.T)


def check_product(g, M, N, K, am=ROW, bm=COL, a_tile=False, b_tile=True, out=F32, bias=False,
                  seed=0, ldc_pad=0, **kw):
    rng = np.random.default_rng(seed + M * 7 + N * 3 + K)
    A, a = operand(g, rng, M, K, am == ROW, a_tile, **kw)
    Bm, b = operand(g, rng, N, K, bm == COL, b_tile, **kw)
    bt = normal(rng, N).float() if bias else None
    buf = torch.full((M, N + ldc_pad), -7.0, dtype=out, device="cuda")
    g.fp8_run(A, Bm, buf[:, :N], bt.cuda() if bias else None, am, bm)
    g.status()
    want = a @ b.T + (bt.double().numpy() if bias else 0.0)
    bound = R.product_bound(a, b.T, want, out)
    if bias:
        bound = bound + 2 * R.U32 * (np.abs(want) + np.abs(bt.double().numpy()))
    err = np.abs(R.host(buf[:, :N]) - want)
    assert (err <= bound).all(), (float((err / bound).max()), int((~(err <= bound)).sum()))
    if ldc_pad:
        assert bool((buf[:, N:] == -7.0).all())


SIZES = [(1, 1, 1), (1, 16, 16), (1, 130, 128), (2, 256, 129), (5, 300, 1000), (16, 512, 2048),
         (17, 129, 640), (33, 1000, 257), (64, 640, 1536), (65, 200, 384), (128, 128, 128),
         (129, 257, 300), (250, 520, 700), (256, 256, 512), (300, 1100, 1024), (777, 900, 200)]


@pytest.mark.parametrize("am,bm", [(ROW, COL), (ROW, ROW), (COL, COL), (COL, ROW)])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product_layouts(g, M, N, K, am, bm):
    check_product(g, M, N, K, am, bm, b_tile=True)
    check_product(g, M, N, K, am, bm, b_tile=False, seed=1)


@pytest.mark.parametrize("a_tile,b_tile", [(True, True), (True, False)])
@pytest.mark.parametrize("M,N,K", [(3, 500, 400), (200, 300, 260), (600, 700, 512)])
def test_product_tile_scales_on_a(g, M, N, K, a_tile, b_tile):
    check_product(g, M, N, K, ROW, COL, a_tile, b_tile)
    check_product(g, M, N, K, COL, ROW, a_tile, b_tile)


@pytest.mark.parametrize("out", [F16, BF16, F32])
@pytest.mark.parametrize("M,N,K", [(1, 333, 512), (40, 129, 300), (300, 513, 700),
                                   (513, 1030, 384)])
def test_product_outputs_bias_and_pitch(g, M, N, K, out):
    check_product(g, M, N, K, out=out, bias=True)
    check_product(g, M, N, K, out=out, bias=True, ldc_pad=3, seed=2)
    check_product(g, M, N, K, out=out, ldc_pad=16, b_tile=False, seed=3)


@pytest.mark.parametrize("M,N,K", [(1, 70, 200), (50, 300, 520), (270, 300, 520)])
def test_product_strides(g, M, N, K):
    """Padded rows (NaN between them), row-major scales, unaligned rows and bases."""
    check_product(g, M, N, K, pad=32)
    check_product(g, M, N, K, pad=16, row_scales=True)
    check_product(g, M, N, K, COL, ROW, pad=16, row_scales=True, b_tile=False)
    check_product(g, M, N, K, pad=5)
    check_product(g, M, N, K, COL, ROW, offset=3)


def test_product_empty(g):
    A = Fp8Matrix.empty(0, 64, "row", "cuda")
    W = Fp8Matrix.empty(32, 64, "tile", "cuda")
    assert g.fp8_matmul(A, W, b_major=COL).shape == (0, 32)
    A = Fp8Matrix.empty(5, 0, "row", "cuda")
    W = Fp8Matrix.empty(32, 0, "tile", "cuda")
    bias = torch.arange(32, dtype=F32, device="cuda")
    assert torch.equal(g.fp8_matmul(A, W, bias, b_major=COL, out_dtype=F32),
                       bias.expand(5, 32))
    assert bool((g.fp8_matmul(A, W, b_major=COL, out_dtype=F32) == 0).all())


@pytest.mark.parametrize("M", [4, 40, 200, 400])
def test_product_nan_stays_in_its_row(g, M):
    rng = np.random.default_rng(M)
    A, a = operand(g, rng, M, 512, True, False)
    W, w = operand(g, rng, 384, 512, True, True)
    A.data[2, 100] = 0x7f
    C = g.fp8_matmul(A, W, b_major=COL, out_dtype=F32)
    nan = torch.isnan(C)
    assert bool(nan[2].all()) and int(nan.sum()) == 384


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (64, 4096, 4096), (200, 1000, 3000),
                                   (1024, 2048, 1024)])
def test_product_repeats_bitwise(g, M, N, K):
    rng = np.random.default_rng(3)
    A, _ = operand(g, rng, M, K, True, False)
    W, _ = operand(g, rng, N, K, True, True)
    first = g.fp8_matmul(A, W, b_major=COL, out_dtype=F32)
    for _ in range(5):
        assert torch.equal(first, g.fp8_matmul(A, W, b_major=COL, out_dtype=F32))
    g.status()


def test_product_long_rows_pass_32_bits(g):
    """Element offsets beyond 2^32 in A and C: the last rows of a tall product."""
    M, N, K = 70000, 64, 128
    ld = 1 << 16  # 64 KiB a row: the last row starts at 4.6e9 bytes
    buf = torch.empty(M * ld, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(5)
    x = normal(rng, 256, K).float()
    q, s = R.quantize(x.numpy(), "row")
    data = torch.as_strided(buf, (M, K), (ld, 1))
    scale = torch.ones(1, M, device="cuda").t()
    data.zero_()
    data[-256:] = torch.from_numpy(q).float().to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    scale[-256:] = torch.from_numpy(s).cuda()
    W, w = operand(g, rng, N, K, True, True)
    cbuf = torch.empty(M * (1 << 16), dtype=F16, device="cuda")
    C = torch.as_strided(cbuf, (M, N), (1 << 16, 1))
    g.fp8_run(Fp8Matrix(data, scale, "row"), W, C, None, ROW, COL)
    g.status()
    a = R.values(q, s, "row")
    want = a @ w.T
    assert (np.abs(R.host(C[-256:]) - want) <= R.product_bound(a, w.T, want, F16)).all()
    assert bool((C[:-256] == 0).all())


def test_other_stream_and_graph(g):
    rng = np.random.default_rng(11)
    x = normal(rng, 96, 512).half().cuda()
    w = g.fp8_quantize(normal(rng, 640, 512).half().cuda(), "tile")
    want = g.fp8_matmul(g.fp8_quantize(x, "row"), w, b_major=COL)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = g.fp8_matmul(g.fp8_quantize(x, "row", stream=s), w, b_major=COL, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = g.fp8_matmul(g.fp8_quantize(x, "row"), w, b_major=COL)
    x.mul_(2)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want * 2)


# -------------------------------------------------------------------- linear --
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,N,K", [(1, 64, 128), (37, 200, 300), (300, 515, 256)])
def test_linear_step_against_formula(g, T, N, K, dtype):
    rng = np.random.default_rng(T + N)
    x = normal(rng, T, K).to(dtype).cuda()
    w = (normal(rng, N, K) * K ** -0.5).to(dtype).cuda()
    dy = normal(rng, T, N).to(dtype).cuda()
    y, saved = fp8.linear_forward(g, x, w)
    dx, dw = fp8.linear_backward(g, dy, saved)

    def q(t, blocks):
        return R.values(*R.quantize(R.host(t), blocks), blocks)

    for got, a, b, odt in ((y, q(x, "row"), q(w, "tile").T, dtype),
                           (dx, q(dy, "row"), q(w, "tile"), dtype),
                           (dw, q(dy, "col").T, q(x, "col"), F32)):
        want = a @ b
        assert got.dtype == odt
        assert (np.abs(R.host(got) - want) <= R.product_bound(a, b, want, odt)).all()


def test_linear_gradient_against_differences(g):
    """The autograd function's gradients of a loss, against central differences
    of the 64-bit loss with the quantisation passed straight through: the loss
    is linear in each of x and w, so a difference of any step is its derivative.
    Powers of two quantise exactly, so nothing but the products is rounded."""
    rng = np.random.default_rng(2)
    T, N, K = 9, 70, 140
    pw = lambda *s: torch.from_numpy(np.exp2(rng.integers(-2, 3, s)) * rng.choice([-1, 1], s))  # noqa: E731
    x, w, c = (pw(T, K).float().cuda().requires_grad_(), pw(N, K).float().cuda().requires_grad_(),
               pw(T, N).float().cuda())
    bias = torch.zeros(N, device="cuda", requires_grad=True)
    (fp8.linear(g, x, w, bias) * c).sum().backward()
    X, W, Cc = R.host(x), R.host(w), R.host(c)

    def loss(X, W):
        return ((X @ W.T) * Cc).sum()

    for t, V, f in ((x, X, lambda V: loss(V, W)), (w, W, lambda V: loss(X, V))):
        for _ in range(12):
            i, j = rng.integers(V.shape[0]), rng.integers(V.shape[1])
            d = np.zeros_like(V)
            d[i, j] = 0.5
            want = f(V + d) - f(V - d)
            assert abs(float(t.grad[i, j]) - want) <= 1e-5 * np.abs(Cc).sum()
    assert np.allclose(R.host(bias.grad), Cc.sum(0), rtol=0, atol=T * R.U32 * np.abs(Cc).sum())


# ----------------------------------------------------------------------- moe --
def expert_weights(rng, E, rows, cols, pad=0):
    q = R.round_e4m3(np.clip(rng.standard_normal((E, rows, cols)) * 112, -448, 448))
    s = ((0.5 + rng.random((E, -(-rows // 128), -(-cols // 128)))) / (112 * cols ** 0.5)
         ).astype(np.float32)
    ld = -(-cols // 16) * 16 + pad
    buf = torch.full((E, rows, ld), 0x7f, dtype=torch.uint8)
    buf[:, :, :cols] = torch.from_numpy(q).float().to(torch.float8_e4m3fn).view(torch.uint8)
    m = Fp8Matrix(buf.cuda()[:, :, :cols], torch.from_numpy(s).cuda(), "tile")
    return m, R.values(q, s, "tile")


def check_moe(g, T, H, I, E, k, dtype=BF16, renorm=True, pad=0, seed=0, skew=0.0, stream=None):
    rng = np.random.default_rng(seed + 1000 * T + H + I + E)
    base = rng.standard_normal((1, H))
    x = torch.from_numpy(rng.standard_normal((T, H)) + skew * base).to(dtype)
    router = torch.from_numpy(rng.standard_normal((E, H)) * H ** -0.5).to(dtype)
    (W1, w1), (W3, w3), (W2, w2) = (expert_weights(rng, E, *s, pad=pad)
                                    for s in ((I, H), (I, H), (H, I)))
    xg = torch.full((T, H + 8), float("nan"), dtype=dtype, device="cuda")
    xg[:, :H] = x.cuda()
    torch.cuda.synchronize()
    out, gi, gg = g.moe_fp8(xg[:, :H], router.cuda(), W1, W3, W2, k, renorm)
    g.status()
    ids = gi.cpu().numpy().astype(np.int64)
    R.check_choice(R.host(x), R.host(router), ids)
    want, slack, gates, e_g = R.moe(R.host(x), R.host(router), w1, w3, w2, ids, renorm)
    assert (np.abs(R.host(gg) - gates) <= e_g).all()
    bound = slack + R.OUT_U[dtype] * (np.abs(want) + slack) + R.OUT_TINY[dtype]
    err = np.abs(R.host(out) - want)
    assert (err <= bound).all(), float((err / bound).max())
    return out


@pytest.mark.parametrize("T,H,I,E,k", [(1, 16, 16, 1, 1), (1, 512, 256, 8, 2), (2, 128, 128, 4, 4),
                                       (3, 1000, 700, 10, 3), (7, 272, 144, 60, 6),
                                       (16, 640, 320, 16, 8), (17, 256, 384, 5, 5),
                                       (33, 384, 200, 3, 1), (64, 256, 256, 4, 2),
                                       (64, 130, 100, 130, 16)])
def test_moe(g, T, H, I, E, k):
    check_moe(g, T, H, I, E, k)
    check_moe(g, T, H, I, E, k, F16, renorm=False, pad=16, seed=1)


def test_moe_all_tokens_to_the_same_experts(g):
    """A router that sends every token to the same experts (one long list, most
    experts empty), and one expert whose every token is the only one."""
    check_moe(g, 64, 256, 256, 32, 2, skew=8.0)
    check_moe(g, 1, 256, 256, 300, 1)


def test_moe_ties_take_the_lowest_index(g):
    rng = np.random.default_rng(1)
    T, H, I, E, k = 5, 256, 128, 12, 4
    (W1, _), (W3, _), (W2, _) = (expert_weights(rng, E, *s) for s in ((I, H), (I, H), (H, I)))
    x = torch.ones(T, H, dtype=BF16, device="cuda")
    x[3] = float("nan")
    router = torch.zeros(E, H, dtype=BF16, device="cuda")
    router[7] = 1.0
    router[2] = -1.0
    out, ids, gates = g.moe_fp8(x, router, W1, W3, W2, k)
    g.status()
    assert ids[[0, 1, 2, 4]].tolist() == [[7, 0, 1, 3]] * 4
    assert ids[3].tolist() == [0, 1, 2, 3]  # every logit NaN: still k different experts
    assert bool(torch.isnan(out[3].float()).all())
    assert not bool(torch.isnan(out[[0, 1, 2, 4]].float()).any())


def test_moe_empty_repeat_and_graph(g):
    rng = np.random.default_rng(4)
    T, H, I, E, k = 9, 512, 256, 16, 4
    (W1, _), (W3, _), (W2, _) = (expert_weights(rng, E, *s) for s in ((I, H), (I, H), (H, I)))
    x = normal(rng, T, H).to(BF16).cuda()
    router = normal(rng, E, H).to(BF16).cuda()
    out, ids, gates = g.moe_fp8(x[:0], router, W1, W3, W2, k)
    assert out.shape == (0, H) and ids.shape == (0, k)
    first = g.moe_fp8(x, router, W1, W3, W2, k)
    for _ in range(20):
        for a, b in zip(first, g.moe_fp8(x, router, W1, W3, W2, k)):
            assert torch.equal(a, b)
    # a token's row does not depend on its neighbours in the batch
    alone = g.moe_fp8(x[4:5], router, W1, W3, W2, k)
    assert torch.equal(alone[1], first[1][4:5])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = g.moe_fp8(x, router, W1, W3, W2, k)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, got):
        assert torch.equal(a, b)
    g.status()


# ------------------------------------------------------------------ refusals --
def test_refusals(g):
    x = torch.zeros(4, 64, dtype=F16, device="cuda")
    W = g.fp8_quantize(torch.zeros(32, 64, device="cuda"), "tile")
    A = g.fp8_quantize(x, "row")
    with pytest.raises(TypeError):
        g.fp8_quantize(x.double())
    with pytest.raises(ValueError):
        g.fp8_quantize(x.t(), "row")
    with pytest.raises(ValueError):
        g.fp8_quantize(x, "diagonal")
    with pytest.raises(ValueError):
        g.fp8_quantize(x.cpu(), "row")
    with pytest.raises(ValueError):
        g.fp8_matmul(A, W)                               # inner sizes differ
    with pytest.raises(B.GemmError) as e:                # blocks do not run along K
        g.fp8_matmul(g.fp8_quantize(x, "col"), W, b_major=COL)
    assert e.value.code == B.GEMM_ERR_INVALID_ARG
    with pytest.raises(TypeError):
        g.fp8_matmul(A, W, b_major=COL, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        g.fp8_matmul(A, W, torch.zeros(31, device="cuda"), b_major=COL)
    E, H, I = 4, 64, 32
    rng = np.random.default_rng(0)
    W1, W3, W2 = (expert_weights(rng, E, *s)[0] for s in ((I, H), (I, H), (H, I)))
    router = torch.zeros(E, H, dtype=F16, device="cuda")
    for bad in (0, E + 1):
        with pytest.raises(ValueError):
            g.moe_fp8(x, router, W1, W3, W2, bad)
    with pytest.raises(ValueError):
        g.moe_fp8(x, router, W1, W2, W3, 1)
    with pytest.raises(TypeError):
        g.moe_fp8(x.float(), router.float(), W1, W3, W2, 1)
    with pytest.raises(B.GemmError) as e:
        g.moe_fp8(torch.zeros(65, H, dtype=F16, device="cuda"), router, W1, W3, W2, 1)
    assert e.value.code == B.GEMM_ERR_UNSUPPORTED
    g.status()


# ------------------------------------------------- splits, chunks and time-outs --
@pytest.mark.parametrize("split", [0, 2, 4, 8])
@pytest.mark.parametrize("M,N,K", [(1, 130, 1100), (20, 300, 1024), (50, 257, 1300),
                                   (100, 200, 2000), (150, 130, 1025)])
def test_product_forced_cluster_splits(g, M, N, K, split):
    """Every cluster size (and none) on ragged tiles, transposed and not."""
    g.set_option(B.GEMM_OPT_CLUSTER_SPLIT, split)
    try:
        check_product(g, M, N, K, bias=True)
        check_product(g, M, N, K, COL, ROW, b_tile=False, out=F16, ldc_pad=1)
    finally:
        g.set_option(B.GEMM_OPT_CLUSTER_SPLIT, -1)


@pytest.mark.parametrize("out,pad", [(F16, 0), (BF16, 4), (F32, 0), (F32, 4), (F16, 3), (F32, 1)])
@pytest.mark.parametrize("am,bm,b_tile", [(ROW, COL, True), (COL, ROW, False)])
@pytest.mark.parametrize("M,N,K", [(2600, 2100, 300), (1281, 5000, 516), (2500, 2136, 257)])
def test_product_wide_tiles(g, M, N, K, am, bm, b_tile, out, pad):
    """More 256-wide tiles than SMs, ragged on both edges, with C whose rows the
    TMA can store and C whose rows it cannot; bytes past N stay."""
    check_product(g, M, N, K, am, bm, b_tile=b_tile, out=out, bias=pad > 0, ldc_pad=pad)


@pytest.mark.parametrize("T,H,I,E,k", [(2, 2304, 2200, 3, 2), (40, 1300, 700, 2, 1),
                                       (64, 1100, 900, 1, 1), (50, 1200, 130, 2, 2),
                                       (3, 256, 4500, 2, 1)])
def test_moe_long_axes_in_pieces(g, T, H, I, E, k):
    """More k-blocks than an operand buffer holds, at each of its widths."""
    check_moe(g, T, H, I, E, k)


@pytest.mark.parametrize("T,H,I,E,k", [(1, 16, 16, 1, 1), (3, 1000, 700, 10, 3), (2, 2304, 2200, 3, 2),
                                       (5, 8400, 130, 4, 2), (3, 256, 8500, 2, 1),
                                       (64, 1100, 900, 3, 2), (64, 130, 100, 130, 16)])
def test_moe_pieces_handed_out_at_run_time(g, T, H, I, E, k):
    """Tiles cut into pieces and pieces of several tiles, forced on work that would
    be cut into equal ranges; the same bits every time."""
    g.set_option(B.GEMM_OPT_DYNAMIC_TILES, 1)
    try:
        first = check_moe(g, T, H, I, E, k)
        for _ in range(3):
            assert torch.equal(first, check_moe(g, T, H, I, E, k))
    finally:
        g.set_option(B.GEMM_OPT_DYNAMIC_TILES, -1)


def test_moe_many_pieces(g):
    """Enough work that pieces are handed out at run time in both phases."""
    first = check_moe(g, 60, 1700, 1300, 64, 2)
    assert torch.equal(first, check_moe(g, 60, 1700, 1300, 64, 2))


def test_moe_scale_strides_and_unaligned_activations(g):
    """Weight scales stored in another order, rows of x and the router that no
    16-byte load can read."""
    rng = np.random.default_rng(8)
    T, H, I, E, k = 4, 300, 260, 6, 3
    ws, vals = [], []
    for s in ((I, H), (I, H), (H, I)):
        m, v = expert_weights(rng, E, *s)
        ws.append(Fp8Matrix(m.data, m.scale.permute(2, 1, 0).contiguous().permute(2, 1, 0), "tile"))
        vals.append(v)
    flat = normal(rng, T * (H + 1) + 1).to(BF16).cuda()
    x = torch.as_strided(flat, (T, H), (H + 1, 1), 1)
    rflat = (normal(rng, E * (H + 3) + 1) * H ** -0.5).to(BF16).cuda()
    router = torch.as_strided(rflat, (E, H), (H + 3, 1), 1)
    out, ids, gates = g.moe_fp8(x, router, *ws, k)
    g.status()
    ids = ids.cpu().numpy().astype(np.int64)
    R.check_choice(R.host(x), R.host(router), ids)
    want, slack, gv, e_g = R.moe(R.host(x), R.host(router), *vals, ids, True)
    assert (np.abs(R.host(gates) - gv) <= e_g).all()
    bound = slack + R.OUT_U[BF16] * (np.abs(want) + slack) + R.OUT_TINY[BF16]
    assert (np.abs(R.host(out) - want) <= bound).all()


def test_moe_other_stream(g):
    rng = np.random.default_rng(6)
    T, H, I, E, k = 6, 256, 128, 8, 2
    (W1, _), (W3, _), (W2, _) = (expert_weights(rng, E, *s) for s in ((I, H), (I, H), (H, I)))
    x, router = normal(rng, T, H).half().cuda(), normal(rng, E, H).half().cuda()
    want = g.moe_fp8(x, router, W1, W3, W2, k)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = g.moe_fp8(x, router, W1, W3, W2, k, stream=s)
    s.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_temporaries_belong_to_the_call_s_stream(g):
    """linear_backward on a busy stream: the quantised dy that it drops must not
    be handed to the current stream's next tensors while that stream is behind."""
    rng = np.random.default_rng(17)
    x, w, dy = (normal(rng, *s).to(BF16).cuda() for s in ((256, 512), (384, 512), (256, 384)))
    y, saved = fp8.linear_forward(g, x, w)
    dx, dw = fp8.linear_backward(g, dy, saved)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        got = fp8.linear_backward(g, dy, saved, stream=s)
        junk = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")
                for n in (256 * 384, 256 * 384 * 2, 4 * 256 * 3, 4 * 2 * 384) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
        del junk
    g.status()


def test_wait_limit_is_reported_and_the_handle_recovers():
    """With a limit of a nanosecond the expert layer's grid barriers give up: the
    launch ends, gemm_status says so, and the handle works again.  A product
    either finishes right or is reported."""
    h = Gemm(torch.device("cuda", 0))
    rng = np.random.default_rng(12)
    T, H, I, E, k = 16, 1024, 512, 16, 4
    (W1, _), (W3, _), (W2, _) = (expert_weights(rng, E, *s) for s in ((I, H), (I, H), (H, I)))
    x, router = normal(rng, T, H).half().cuda(), normal(rng, E, H).half().cuda()
    want = h.moe_fp8(x, router, W1, W3, W2, k)
    h.status()
    s = torch.cuda.current_stream().cuda_stream
    h.set_option(B.GEMM_OPT_WAIT_LIMIT_NS, 1)
    h.moe_fp8(x, router, W1, W3, W2, k)
    assert B.gemm_status(h.handle, s) == B.GEMM_ERR_DEVICE_TIMEOUT
    A = h.fp8_quantize(normal(rng, 300, 2048).half().cuda(), "row")
    W = h.fp8_quantize(normal(rng, 700, 2048).half().cuda(), "tile")
    C = h.fp8_matmul(A, W, b_major=COL, out_dtype=F32)
    rc = B.gemm_status(h.handle, s)
    assert rc in (B.GEMM_OK, B.GEMM_ERR_DEVICE_TIMEOUT)
    h.set_option(B.GEMM_OPT_WAIT_LIMIT_NS, -1)
    again = h.fp8_matmul(A, W, b_major=COL, out_dtype=F32)
    if rc == B.GEMM_OK:
        assert torch.equal(C, again)
    for a, b in zip(want, h.moe_fp8(x, router, W1, W3, W2, k)):
        assert torch.equal(a, b)
    h.status()
    h.close()


def test_example_trains_and_serves(capsys):
    import os
    import runpy
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "fp8_layers.py")
    losses, off, drift = runpy.run_path(path)["main"](["--hidden", "256", "--steps", "12"])
    # 8 bits keep about 4 % of an operand's elements' size as noise
    assert losses[-1] < 0.1 * losses[0] and off < 0.3 and drift < 0.02
