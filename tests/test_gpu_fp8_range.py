"""Scales whose product leaves fp32's range where the term it belongs to does not:
block maxima of 1e30 against 1e14 where one operand is zero, products below the
smallest normal number, and products above the largest of sums below 1.  Every
kernel of the block-scaled product, and the expert layer."""
import numpy as np
import pytest
import torch

import fp8_reference as R
from dense_gemm_tmem_gb300 import binding as B
from dense_gemm_tmem_gb300.fp8 import Fp8Matrix
from dense_gemm_tmem_gb300.gemm import COL, ROW, Gemm

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    h = Gemm(torch.device("cuda", 0))
    yield h
    h.close()


def stored(values, scales, blocks, pad=0):
    """e4m3 values and scales (arrays) as an Fp8Matrix, rows padded to 16 bytes and
    by `pad` more, and the doubles they stand for."""
    r, c = values.shape
    buf = torch.zeros(r, -(-c // 16) * 16 + pad, dtype=torch.uint8)
    buf[:, :c] = torch.from_numpy(values).float().to(torch.float8_e4m3fn).view(torch.uint8)
    s = torch.from_numpy(scales.astype(np.float32))
    return (Fp8Matrix(buf.cuda()[:, :c], s.cuda(), blocks),
            R.values(values, scales.astype(np.float32), blocks))


def operand(rng, mn, K, k_rows, tile, factor, fill, pad):
    """Values by fill(mn, K); block scales around factor[kb]."""
    blocks = "tile" if tile else ("row" if k_rows else "col")
    v = fill(mn, K) if k_rows else fill(mn, K).T
    v = np.ascontiguousarray(v)
    br, bc = R.SHAPE[blocks]
    s = 0.5 + rng.random((-(-v.shape[0] // br), -(-v.shape[1] // bc)))
    f = np.asarray(factor, np.float64)[:s.shape[1 if k_rows else 0]]
    s = s * (f[None, :] if k_rows else f[:, None])
    m, x = stored(v, s, blocks, pad)
    return m, (x if k_rows else x.T)


# transposed of 32, 64 and 128 columns, split and not; 64, 128 and 256 wide; unaligned
SHAPES = [(1, 300, 1280, 0), (40, 1100, 640, 0), (100, 2000, 640, 0), (200, 700, 650, 0),
          (520, 4096, 640, 0), (2600, 2100, 640, 0), (50, 70, 640, 5)]
LAYOUTS = [(ROW, COL, False, True), (ROW, COL, False, False), (COL, ROW, False, False),
           (ROW, ROW, True, True)]


def check(g, rng, shape, layout, fa, fb, fill_a, fill_b):
    M, N, K, pad = shape
    am, bm, a_tile, b_tile = layout
    A, a = operand(rng, M, K, am == ROW, a_tile, fa, fill_a, pad)
    W, b = operand(rng, N, K, bm == COL, b_tile, fb, fill_b, pad)
    got = R.host(g.fp8_matmul(A, W, a_major=am, b_major=bm, out_dtype=F32))
    g.status()
    want = a @ b.T
    # a k-block's term is rounded once more, and to no less than the smallest number
    bound = R.product_bound(a, b.T, want, F32) * (1 + 1 / 64) + 2.0 ** -149 * (-(-K // 128) + 1)
    assert np.isfinite(want).all() and np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= bound).all(), float((err / bound).max())


def signs(rng):
    return lambda mn, K: R.round_e4m3(np.clip(rng.standard_normal((mn, K)) * 100, -448, 448))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("shape", SHAPES)
def test_overflowing_scales_of_zero_sums(g, shape, layout):
    """1e30 and 1e14 in the same k-blocks, the operands zero in opposite halves of
    them; the other k-blocks are ordinary."""
    rng = np.random.default_rng(1)
    kb = -(-shape[2] // 128)
    hot = np.arange(kb) % 3 == 1
    fa, fb = np.where(hot, 1e30 / 448, 1.0), np.where(hot, 1e14 / 448, 1.0)

    def half(lower):
        def fill(mn, K):
            v = signs(rng)(mn, K)
            k = np.arange(K)
            v[:, hot[k // 128] & ((k % 128 < 64) == lower)] = 0.0
            return v
        return fill

    check(g, rng, shape, layout, fa, fb, half(True), half(False))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("shape", SHAPES)
def test_subnormal_scale_products(g, shape, layout):
    """Scale products around 2^-142 (seven bits left) under sums of 2^21."""
    rng = np.random.default_rng(2)
    kb = -(-shape[2] // 128)
    fill = lambda mn, K: R.round_e4m3(100 + 200 * rng.random((mn, K)))  # noqa: E731
    check(g, rng, shape, layout, np.full(kb, 2.0 ** -80), np.full(kb, 2.0 ** -62), fill, fill)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("shape", SHAPES)
def test_overflowing_scale_products_of_small_sums(g, shape, layout):
    """Scale products of 2^134 over sums of 2^-11: terms of 2^123.  Blocks of zeros
    as the quantiser stores them (the smallest scale it makes) between them."""
    rng = np.random.default_rng(3)
    kb = -(-shape[2] // 128)
    fa = np.where(np.arange(kb) == 2, 2.0 ** -100 / 448, 2.0 ** 69)
    fb = np.full(kb, 2.0 ** 65)

    def fill(zero):
        def f(mn, K):
            v = np.full((mn, K), 2.0 ** -9)
            if zero:
                v[:, 256:384] = 0.0
            return v
        return f

    check(g, rng, shape, layout, fa, fb, fill(True), fill(False))


@pytest.mark.parametrize("fa,fb", [(2.0 ** 112, 2.0 ** -105), (2.0 ** -105, 2.0 ** 112)])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("shape", SHAPES)
def test_scales_from_both_ends(g, shape, layout, fa, fb):
    """Scales of 2^112 (block maxima of 2e36) against 2^-105 in some k-blocks, ordinary
    ones in the others, terms of the same size."""
    rng = np.random.default_rng(4)
    hot = np.arange(-(-shape[2] // 128)) % 2 == 1
    check(g, rng, shape, layout, np.where(hot, fa, 1.0), np.where(hot, fb, 2.0 ** 7), signs(rng),
          signs(rng))


@pytest.mark.parametrize("T,H,I,E,k", [(1, 512, 256, 4, 2), (5, 640, 300, 4, 3),
                                       (40, 2304, 256, 2, 1)])
def test_expert_layer(g, T, H, I, E, k):
    """Token blocks of 1e30 against weight scales of 1e14 where the weights are zero,
    and tokens of zeros (padding) beside them."""
    rng = np.random.default_rng(T)
    x = rng.standard_normal((T, H))
    x[:, 128:256] *= 1e30
    if T > 1:
        x[1] = 0.0
    x = torch.from_numpy(x).to(BF16)
    router = rng.standard_normal((E, H)) * H ** -0.5
    router[:, 128:256] = 0.0
    router = torch.from_numpy(router).to(BF16)

    def weights(rows, cols, first):
        v = R.round_e4m3(np.clip(rng.standard_normal((E, rows, cols)) * 112, -448, 448))
        s = (0.5 + rng.random((E, -(-rows // 128), -(-cols // 128)))) / (112 * cols ** 0.5)
        if first:
            v[:, :, 128:256] = 0.0
            s[:, :, 1] = 1e14
        ld = -(-cols // 16) * 16
        buf = torch.zeros(E, rows, ld, dtype=torch.uint8)
        buf[:, :, :cols] = torch.from_numpy(v).float().to(torch.float8_e4m3fn).view(torch.uint8)
        s = s.astype(np.float32)
        return (Fp8Matrix(buf.cuda()[:, :, :cols], torch.from_numpy(s).cuda(), "tile"),
                R.values(v, s, "tile"))

    (W1, w1), (W3, w3), (W2, w2) = weights(I, H, True), weights(I, H, True), weights(H, I, False)
    out, ids, gates = g.moe_fp8(x.cuda(), router.cuda(), W1, W3, W2, k)
    g.status()
    ids = ids.cpu().numpy().astype(np.int64)
    R.check_choice(R.host(x), R.host(router), ids)
    want, slack, gv, e_g = R.moe(R.host(x), R.host(router), w1, w3, w2, ids, True)
    assert (np.abs(R.host(gates) - gv) <= e_g).all()
    got = R.host(out)
    assert np.isfinite(got).all()
    bound = slack + R.OUT_U[BF16] * (np.abs(want) + slack) + R.OUT_TINY[BF16]
    assert (np.abs(got - want) <= bound).all()


def test_quantised_matrices(g):
    """The same through the quantiser: columns of 1e30 against rows of 1e14, each
    where the other matrix is zero."""
    rng = np.random.default_rng(9)
    x = torch.from_numpy(rng.standard_normal((70, 512))).float()
    w = torch.from_numpy(rng.standard_normal((300, 512))).float()
    x[:, 130:140] = 1e30
    w[:, 130:140] = 0.0
    w[:, 150:160] = 1e14
    x[:, 150:160] = 0.0
    xq, wq = g.fp8_quantize(x.cuda(), "row"), g.fp8_quantize(w.cuda(), "tile")
    got = R.host(g.fp8_matmul(xq, wq, b_major=COL, out_dtype=F32))
    a = R.values(*R.quantize(x.numpy(), "row"), "row")
    b = R.values(*R.quantize(w.numpy(), "tile"), "tile")
    want = a @ b.T
    assert (np.abs(got - want) <= R.product_bound(a, b.T, want, F32) * (1 + 1 / 64)).all()
