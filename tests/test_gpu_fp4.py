"""The 4-bit operators on the GPU against a 64-bit reference: quantising bit for bit,
reading back and products within bounds derived from their fp32 arithmetic, at the
sizes, strides and values where they can go wrong."""
import numpy as np
import pytest
import torch

import fp4_reference as R
from dense_gemm_tmem_gb300 import binding as B
from dense_gemm_tmem_gb300 import fp4
from dense_gemm_tmem_gb300.fp4 import Fp4Matrix
from dense_gemm_tmem_gb300.gemm import Gemm

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
FORMATS = ["mxfp4", "nvfp4"]


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    h = Gemm(torch.device("cuda", 0))
    yield h
    h.close()


def host(t):
    return t.double().cpu().numpy()


def make(rng, rows, cols, spread=1.0):
    return torch.from_numpy(rng.standard_normal((rows, cols))
                            * np.exp(spread * rng.standard_normal((1, cols))))


def check_quantized(m, x, fmt):
    code, byte, rows = R.quantize(host(x), fmt)
    got_code, got_byte = R.stored(m)
    assert np.array_equal(got_byte, byte), int((got_byte != byte).sum())
    assert np.array_equal(got_code, code), int((got_code != code).sum())
    if rows is None:
        assert m.row_scale is None
    else:
        assert np.array_equal(host(m.row_scale), rows)
    # every byte of a piece past the matrix is 0, and so is the odd column's partner
    blocks = byte.shape[1]
    full = np.zeros(m.scale.numel(), np.uint8)
    r, b = np.arange(m.shape[0])[:, None], np.arange(blocks)[None, :]
    full[R.place(r, b, blocks)] = byte
    assert np.array_equal(m.scale.cpu().numpy(), full)
    assert np.array_equal(m.data.cpu().numpy(), R.pack(code))


# ------------------------------------------------------------------ quantise --
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 16), (3, 33), (128, 64), (129, 127), (5, 1025),
                                       (260, 1000), (1, 4096), (2, 8192), (2, 8209), (3, 20001)])
def test_quantize(g, rows, cols, dtype, fmt):
    rng = np.random.default_rng(rows * 1000 + cols)
    x = make(rng, rows, cols).to(dtype).cuda()
    check_quantized(g.fp4_quantize(x, fmt), x, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_quantize_values_at_the_ends(g, dtype, fmt):
    """Zeros, a type's largest and smallest, ties, infinities and NaN, rows of them."""
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal / 4
    x = torch.zeros(12, 96, dtype=dtype)
    x[1] = big
    x[2] = tiny
    x[3, 5], x[3, 70] = float("inf"), float("nan")
    x[3, 40] = -2.5
    x[4, 0::2] = 6.0  # block maximum 6: scales of powers of two, every tie of e2m1 below
    x[4, 1:32:2] = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5,
                                 -3.5, -5, .2, -.2], dtype=dtype)
    x[5, 0], x[5, 50] = big, tiny
    x[6] = -0.0
    x[7, 33] = tiny
    x[8] = float("-inf")
    x[9] = torch.linspace(-7, 7, 96).to(dtype)
    x[10, 17] = big
    x[10, 18] = float("nan")
    x[11] = torch.linspace(0, 1, 96).to(dtype) ** 8
    x = x.cuda()
    check_quantized(g.fp4_quantize(x, fmt), x, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offset,pitch", [(1, 401), (8, 408), (0, 403), (3, 440), (5, 390),
                                          (6, 396), (7, 391)])
def test_quantize_strided_rows(g, dtype, fmt, offset, pitch):
    rng = np.random.default_rng(offset)
    buf = make(rng, 37, 450).to(dtype).cuda().reshape(-1)
    x = torch.as_strided(buf, (37, 390), (pitch, 1), offset)
    check_quantized(g.fp4_quantize(x, fmt), x, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_leaves_the_padding_of_rows(g, fmt):
    rows, cols = 5, 45  # 23 bytes a row
    buf = torch.full((rows, 32), 0xa5, dtype=torch.uint8, device="cuda")
    scale = torch.empty(fp4.scale_bytes(rows, cols, fmt), dtype=torch.uint8, device="cuda")
    r = torch.empty(2 * rows, device="cuda")[::2] if fmt == "nvfp4" else None
    m = Fp4Matrix(buf[:, :23], scale, r, (rows, cols), fmt)
    x = torch.randn(rows, cols, device="cuda")
    rc = B.gemm_fp4_quantize(g.handle, rows, cols, x.data_ptr(), cols, B.GEMM_F32, m.desc(),
                             torch.cuda.current_stream().cuda_stream)
    assert rc == B.GEMM_OK
    check_quantized(m, x, fmt)
    assert bool((buf[:, 23:] == 0xa5).all())


def test_tokens_do_not_depend_on_each_other(g):
    x = torch.randn(300, 700, device="cuda").bfloat16()
    for fmt in FORMATS:
        all_, one = g.fp4_quantize(x, fmt), g.fp4_quantize(x[177:178], fmt)
        assert torch.equal(all_.data[177:178], one.data)
        assert np.array_equal(R.stored(all_)[1][177:178], R.stored(one)[1])


# ------------------------------------------------------------------ read back --
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (130, 65), (17, 1000), (1, 4096)])
def test_dequantize(g, rows, cols, dtype, fmt):
    rng = np.random.default_rng(rows + cols)
    m = g.fp4_quantize(make(rng, rows, cols).cuda().float(), fmt)
    got, want = g.fp4_dequantize(m, dtype), R.values(m)
    assert got.dtype == dtype and got.shape == (rows, cols)
    # the row scale's product and the last rounding
    tol = np.abs(want) * (2.0 ** -24 + torch.finfo(dtype).eps / 2) + \
        torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    assert np.all(np.abs(host(got) - want) <= tol)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("cols,pitch,offset", [(37, 37, 0), (200, 201, 1), (300, 303, 5),
                                               (64, 72, 3), (9, 11, 7), (2100, 2101, 2)])
def test_dequantize_into_strided_rows(g, dtype, fmt, cols, pitch, offset):
    """Rows that start anywhere, and nothing written beside them."""
    rows = 13
    m = g.fp4_quantize(torch.randn(rows, cols, device="cuda"), fmt)
    buf = torch.full((rows * pitch + offset + 9,), 7.0, dtype=dtype, device="cuda")
    out = torch.as_strided(buf, (rows, cols), (pitch, 1), offset)
    code = B.GEMM_F32 if dtype == F32 else B.GEMM_F16
    assert B.gemm_fp4_dequantize(g.handle, rows, cols, m.desc(), out.data_ptr(), pitch, code,
                                 torch.cuda.current_stream().cuda_stream) == B.GEMM_OK
    assert torch.equal(out, g.fp4_dequantize(m, dtype))
    out.fill_(7.0)
    assert bool((buf == 7.0).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_dequantize_every_code_and_scale(g, fmt):
    """All 16 values under all 256 scale bytes (e4m3's sign bit too), with one scale for the
    matrix and none."""
    n = R.BLOCK[fmt]
    data = torch.arange(n // 2, dtype=torch.int32) % 8
    data = ((2 * data) + 16 * (2 * data + 1)).to(torch.uint8).repeat(256, 1).cuda()
    scale = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(256, 1).cuda()
    for rs in (None, torch.tensor([1.5], device="cuda")):
        m = Fp4Matrix.from_parts(data, scale, rs, n, fmt)
        got, want = host(g.fp4_dequantize(m, F32)), R.values(m)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        ok = np.isfinite(want) & (np.abs(want) < 3e38)
        assert np.array_equal(got[ok], R.f32(want[ok]))


@pytest.mark.parametrize("row", [0.25, -0.3, 1e-30, 2.0 ** -149, 0.0, 1.0, -1.5])
def test_dequantize_the_largest_scales_with_a_row_scale(g, row):
    """Value times block scale may lie beyond fp32 where the row scale brings it back: rows
    that start on 16 bytes, and rows that start anywhere, whose 16 bytes meet two blocks."""
    cols = 96
    data = (torch.arange(48) * 37 % 256).to(torch.uint8).expand(4, 48).contiguous().cuda()
    scale = torch.tensor([[254, 253, 252], [1, 254, 0], [253, 127, 254], [252, 254, 253]],
                         dtype=torch.uint8, device="cuda")
    m = Fp4Matrix.from_parts(data, scale, torch.tensor([row], device="cuda"), cols, "mxfp4")
    want = R.f32(R.values(m))
    assert np.array_equal(host(g.fp4_dequantize(m, F32)), want)
    for pitch, offset in ((97, 3), (98, 1)):
        buf = torch.zeros(4 * pitch + offset, device="cuda")
        out = torch.as_strided(buf, (4, cols), (pitch, 1), offset)
        assert B.gemm_fp4_dequantize(g.handle, 4, cols, m.desc(), out.data_ptr(), pitch, B.GEMM_F32,
                                     torch.cuda.current_stream().cuda_stream) == B.GEMM_OK
        assert np.array_equal(host(out), want)


# -------------------------------------------------------------------- product --
def bound(a, b, ra, rb, want, bias, dtype):
    """Exact products summed in fp32 in any order and with truncating adders lose at most
    2^-23 of the sum of magnitudes per addition; then the two row scales, the bias, each
    rounded, and C's rounding (half a step of its type, subnormals included)."""
    K = a.shape[1]
    mag = np.abs(a) @ np.abs(b).T
    if ra is not None:
        mag = mag * ra[:, None]
    if rb is not None:
        mag = mag * rb[None, :]
    err = mag * (K * 2.0 ** -23 + 2 * 2.0 ** -24) + 2.0 ** -24 * np.abs(want)
    if bias is not None:
        err = err + 2.0 ** -24 * np.abs(bias)[None, :]
    f = torch.finfo(dtype)
    return err + np.abs(want) * f.eps / 2 + f.smallest_normal * f.eps


def parts(m):
    code, byte = R.stored(m)
    rows = None if m.row_scale is None else host(m.row_scale)
    return R.times_blocks(code, byte, m.format), rows


def check_product(C, A, Bm, bias=None):
    (a, ra), (b, rb) = parts(A), parts(Bm)
    want = a @ b.T
    want = want * (1 if ra is None else ra[:, None]) * (1 if rb is None else rb[None, :])
    bias = None if bias is None else host(bias)
    if bias is not None:
        want = want + bias[None, :]
    got = host(C)
    assert got.shape == want.shape
    tol = bound(a, b, ra, rb, want, bias, C.dtype)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - want)[bad].max()),
                           np.argwhere(bad)[:5])


SHAPES = [(1, 1, 1), (1, 16, 16), (1, 128, 64), (2, 3, 5), (5, 130, 63), (128, 128, 256),
          (127, 129, 255), (1, 4096, 4096), (16, 1000, 2056), (33, 520, 777), (64, 300, 100),
          (65, 64, 4100), (129, 1, 300), (257, 260, 512), (300, 700, 1025), (515, 1000, 2056),
          (1001, 514, 260), (256, 512, 64), (1024, 2304, 130)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(g, M, N, K, fmt):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    A = g.fp4_quantize(make(rng, M, K).cuda().float(), fmt)
    Bm = g.fp4_quantize(make(rng, N, K, 0.2).cuda().float(), fmt)
    bias = torch.from_numpy(rng.standard_normal(N)).float().cuda() if (M + N) % 2 else None
    for dtype in (F32, F16, BF16):
        check_product(g.fp4_matmul(A, Bm, bias, out_dtype=dtype), A, Bm, bias)
    g.status()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(2048, 2304, 576), (1600, 4000, 320), (2560, 2816, 2100)])
def test_product_of_many_tiles(g, M, N, K, fmt):
    """Several tiles a CTA; a sample of rows against doubles."""
    rng = np.random.default_rng(M)
    A = g.fp4_quantize(make(rng, M, K).cuda().float(), fmt)
    Bm = g.fp4_quantize(make(rng, N, K).cuda().float(), fmt)
    check_product(g.fp4_matmul(A, Bm, out_dtype=F16), A, Bm)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("swap,tile,split", [(1, -1, 0), (1, -1, 4), (0, 64, 0), (0, 64, 2), (0, 64, 8),
                                             (0, 128, 0), (0, 128, 4), (0, 256, -1)])
@pytest.mark.parametrize("M,N,K", [(1, 130, 2100), (32, 300, 2304), (20, 64, 70), (300, 450, 2500)])
def test_every_tile_on_every_shape(g, M, N, K, swap, tile, split, fmt):
    """What the rule takes elsewhere, forced: swapped operands, tile widths, CTA pairs, splits."""
    rng = np.random.default_rng(M)
    A = g.fp4_quantize(make(rng, M, K).cuda().float(), fmt)
    Bm = g.fp4_quantize(make(rng, N, K).cuda().float(), fmt)
    bias = torch.from_numpy(rng.standard_normal(N)).float().cuda()
    forced = {B.GEMM_OPT_FORCE_SWAP_AB: swap, B.GEMM_OPT_FORCE_TILE_N: tile,
              B.GEMM_OPT_CLUSTER_SPLIT: split}
    try:
        for o, v in forced.items():
            g.set_option(o, v)
        for dtype in (F32, BF16):
            check_product(g.fp4_matmul(A, Bm, bias, out_dtype=dtype), A, Bm, bias)
        g.status()
    finally:
        for o in forced:
            g.set_option(o, -1)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("split", [-1, 0, 2, 4, 8])
@pytest.mark.parametrize("M,N,K", [(33, 150, 2100), (63, 129, 70), (64, 400, 2304), (48, 2100, 2307)])
def test_swapped_in_two_widths(g, M, N, K, split, fmt):
    """33 to 64 rows of A as the MMA's columns."""
    rng = np.random.default_rng(N)
    A = g.fp4_quantize(make(rng, M, K).cuda().float(), fmt)
    Bm = g.fp4_quantize(make(rng, N, K).cuda().float(), fmt)
    bias = torch.from_numpy(rng.standard_normal(N)).float().cuda()
    g.set_option(B.GEMM_OPT_FORCE_SWAP_AB, 1)
    g.set_option(B.GEMM_OPT_CLUSTER_SPLIT, split)
    try:
        for dtype in (F32, F16, BF16):
            buf = torch.full((M, N + 3), 7.0, device="cuda").to(dtype)
            g.fp4_run(A, Bm, buf[:, :N], bias)
            check_product(buf[:, :N], A, Bm, bias)
            assert bool((buf[:, N:] == 7).all())
        g.status()
    finally:
        g.set_option(B.GEMM_OPT_FORCE_SWAP_AB, -1)
        g.set_option(B.GEMM_OPT_CLUSTER_SPLIT, -1)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("K", [257, 1281, 1400, 1537, 1790, 2049])
@pytest.mark.parametrize("M,N", [(1, 300), (3, 64), (70, 200)])
def test_few_tiles_over_few_k_blocks(g, M, N, K, fmt):
    """Fewer k-blocks than CTAs that a tile might be split over."""
    rng = np.random.default_rng(K)
    A = g.fp4_quantize(make(rng, M, K).cuda().float(), fmt)
    Bm = g.fp4_quantize(make(rng, N, K).cuda().float(), fmt)
    for _ in range(3):
        check_product(g.fp4_matmul(A, Bm, out_dtype=F32), A, Bm)
    g.status()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", [(7, 100), (130, 1000), (700, 516)])
def test_a_matrix_by_itself(g, M, K, fmt):
    rng = np.random.default_rng(M)
    A = g.fp4_quantize(make(rng, M, K).cuda().float(), fmt)
    check_product(g.fp4_matmul(A, A, out_dtype=F32), A, A)


@pytest.mark.parametrize("fmt", FORMATS)
def test_without_programmatic_launches(g, fmt):
    """GEMM_OPT_PDL changes when kernels start, and nothing else."""
    rng = np.random.default_rng(11)
    x = make(rng, 33, 520).cuda().float()
    w = g.fp4_quantize(make(rng, 300, 520).cuda().float(), fmt)
    def run():
        q = g.fp4_quantize(x, fmt)
        return q.data, q.scale, g.fp4_linear(x, w), g.fp4_dequantize(q)
    want = run()
    g.set_option(B.GEMM_OPT_PDL, 0)
    try:
        got = run()
    finally:
        g.set_option(B.GEMM_OPT_PDL, -1)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 300, 200), (200, 300, 520), (700, 1024, 256)])
def test_product_into_strided_rows(g, M, N, K, fmt):
    rng = np.random.default_rng(K)
    A = g.fp4_quantize(make(rng, M, K).cuda().float(), fmt)
    Bm = g.fp4_quantize(make(rng, N, K).cuda().float(), fmt)
    for dtype in (F16, F32):
        for offset, pitch in ((0, N), (1, N + 3), (8, N + 8)):
            buf = torch.full((M * pitch + offset + 64,), 7.0, dtype=dtype, device="cuda")
            C = torch.as_strided(buf, (M, N), (pitch, 1), offset)
            g.fp4_run(A, Bm, C)
            check_product(C, A, Bm)
            C.fill_(7.0)
            assert bool((buf == 7.0).all())  # nothing outside C was written


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [1, 40, 300])
def test_scales_at_the_ends_and_nan(g, M, fmt):
    """A NaN scale reaches its row or column of C and nothing else; the largest and smallest
    scales; operands whose rows are padded with bytes that are no part of them."""
    N, K = 260, 320
    n = R.BLOCK[fmt]
    rng = np.random.default_rng(M)

    def operand(rows, lo, hi):
        data = torch.from_numpy(rng.integers(0, 256, (rows, K // 2)).astype(np.uint8)).cuda()
        scale = torch.from_numpy(rng.integers(lo, hi, (rows, K // n)).astype(np.uint8)).cuda()
        buf = torch.full((rows, K // 2 + 32), 0x77, dtype=torch.uint8, device="cuda")
        buf[:, :K // 2] = data
        return buf, scale

    lo, hi = (60, 190) if fmt == "mxfp4" else (0, 127)
    da, sa = operand(M, lo, hi)
    db, sb = operand(N, 100, 128) if fmt == "mxfp4" else operand(N, 0, 127)
    for nan in (False, True):
        if nan:
            sa[M // 2, 3] = 255 if fmt == "mxfp4" else 127
            sb[N - 1, K // n - 1] = 255 if fmt == "mxfp4" else 127
        A = Fp4Matrix(da[:, :K // 2], fp4.pack_scales(sa), None, (M, K), fmt)
        Bm = Fp4Matrix(db[:, :K // 2], fp4.pack_scales(sb), None, (N, K), fmt)
        C = g.fp4_matmul(A, Bm, out_dtype=F32)
        if nan:
            want = torch.zeros(M, N, dtype=torch.bool)
            want[M // 2], want[:, N - 1] = True, True
            assert torch.equal(torch.isnan(C).cpu(), want)
        else:
            check_product(C, A, Bm)


def test_row_scales(g):
    """One for all (stride 0), every second of a tensor, on one side only, in mxfp4 too."""
    rng = np.random.default_rng(0)
    M, N, K = 150, 200, 256
    for fmt in FORMATS:
        A = g.fp4_quantize(make(rng, M, K).cuda().float(), fmt)
        Bm = g.fp4_quantize(make(rng, N, K).cuda().float(), fmt)
        for ra in (None, torch.tensor([0.3], device="cuda").expand(M),
                   torch.rand(2 * M, device="cuda")[::2]):
            A2 = Fp4Matrix(A.data, A.scale, ra, (M, K), fmt)
            check_product(g.fp4_matmul(A2, Bm, out_dtype=F32), A2, Bm)
            check_product(g.fp4_matmul(Bm, A2, out_dtype=F32), Bm, A2)


def test_empty_sizes(g):
    z = lambda r, c, f: g.fp4_quantize(torch.zeros(r, c, device="cuda"), f)  # noqa: E731
    for fmt in FORMATS:
        assert g.fp4_matmul(z(0, 64, fmt), z(5, 64, fmt)).shape == (0, 5)
        assert g.fp4_matmul(z(5, 64, fmt), z(0, 64, fmt)).shape == (5, 0)
        bias = torch.randn(7, device="cuda")
        C = g.fp4_matmul(z(3, 0, fmt), z(7, 0, fmt), bias, out_dtype=F32)
        assert torch.equal(C, bias.expand(3, 7))
        assert float(g.fp4_matmul(z(3, 0, fmt), z(7, 0, fmt), out_dtype=F32).abs().sum()) == 0
        assert g.fp4_dequantize(z(0, 8, fmt)).shape == (0, 8)
        assert g.fp4_linear(torch.zeros(0, 64, device="cuda"), z(5, 64, fmt)).shape == (0, 5)


# ------------------------------------------------------------------ as a user --
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("T,N,K", [(1, 300, 260), (70, 512, 1000), (300, 257, 512)])
def test_linear_is_quantising_and_product(g, T, N, K, dtype, fmt):
    rng = np.random.default_rng(T)
    x = make(rng, T, K).cuda().to(dtype)
    w = g.fp4_quantize(make(rng, N, K).cuda().float(), fmt)
    bias = torch.randn(N, device="cuda")
    for b in (None, bias):
        y = fp4.linear(g, x, w, b)
        assert y.dtype == dtype
        check_product(y, g.fp4_quantize(x, fmt), w, b)


def test_streams_graphs_and_repeats(g):
    """Another stream, a captured and replayed chain, the same bits every time."""
    torch.manual_seed(0)
    for fmt in FORMATS:
        for T in (1, 200, 1030):
            x = torch.randn(T, 1000, device="cuda").bfloat16()
            w = g.fp4_quantize(torch.randn(520, 1000, device="cuda"), fmt)
            want = fp4.linear(g, x, w)
            for _ in range(3):
                assert torch.equal(fp4.linear(g, x, w), want)
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            y = fp4.linear(g, x, w, stream=s)
            q = g.fp4_quantize(x, fmt, stream=s)
            C = g.fp4_matmul(q, w, stream=s)
            back = g.fp4_dequantize(q, stream=s)
            s.synchronize()
            assert torch.equal(y, want) and torch.equal(C, want)
            assert torch.equal(back, g.fp4_dequantize(q))
            graph = torch.cuda.CUDAGraph()
            static = x.clone()
            with torch.cuda.graph(graph):
                out = fp4.linear(g, static, w)
            x2 = torch.randn_like(x)
            static.copy_(x2)
            graph.replay()
            assert torch.equal(out, fp4.linear(g, x2, w))
    g.status()


def test_from_parts_is_what_quantising_stores(g):
    for fmt in FORMATS:
        for rows, cols in ((3, 45), (130, 64), (257, 1000)):
            m = g.fp4_quantize(torch.randn(rows, cols, device="cuda"), fmt)
            again = Fp4Matrix.from_parts(m.data.contiguous(), m.block_scales(), m.row_scale, cols,
                                         fmt)
            assert torch.equal(again.data, m.data) and torch.equal(again.scale, m.scale)


# -------------------------------------------------------------- one row of A --
def codes(rng, rows, cols, fmt, lo, hi):
    """A matrix of any codes, its rows' padding full of bytes that are no part of it, and
    block scales of lo ... hi - 1."""
    width = (cols + 1) // 2
    buf = torch.full((rows, -(-width // 16) * 16 + 16), 0x77, dtype=torch.uint8)
    buf[:, :width] = torch.from_numpy(rng.integers(0, 256, (rows, width)).astype(np.uint8))
    if cols % 2:
        buf[:, width - 1] &= 15
    scale = torch.from_numpy(rng.integers(lo, hi, (rows, -(-cols // R.BLOCK[fmt]))).astype(np.uint8))
    return Fp4Matrix(buf.cuda()[:, :width], fp4.pack_scales(scale.cuda()), None, (rows, cols), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("K", [1, 2, 15, 16, 17, 33, 63, 65, 129, 2047, 2048, 2050, 4100, 10000,
                               32770])
@pytest.mark.parametrize("N", [1, 31, 32, 33, 97, 127, 128, 129, 700])
def test_one_row(g, N, K, fmt):
    rng = np.random.default_rng(N * 7 + K)
    lo, hi = (117, 137) if fmt == "mxfp4" else (0, 127)
    A, Bm = codes(rng, 1, K, fmt, lo, hi), codes(rng, N, K, fmt, lo, hi)
    bias = torch.randn(N, device="cuda") if K % 2 else None
    for dtype in (F32, BF16):
        out = g.fp4_matmul(A, Bm, bias, out_dtype=dtype)
        check_product(out, A, Bm, bias)
        assert torch.equal(g.fp4_matmul(A, Bm, bias, out_dtype=dtype), out)
    # what follows the row stays as it was
    C = torch.full((N + 5,), 7.0, device="cuda")
    g.fp4_run(A, Bm, C[2:N + 2].view(1, N), bias)
    check_product(C[2:N + 2].view(1, N), A, Bm, bias)
    assert bool((C[:2] == 7).all()) and bool((C[N + 2:] == 7).all())


@pytest.mark.parametrize("N,K", [(40000, 520), (14336, 2048), (300, 40000)])
def test_one_row_of_many(g, N, K):
    """More rows than are resident at once, and parts of K that several rounds take."""
    for fmt in FORMATS:
        rng = np.random.default_rng(K)
        lo, hi = (117, 137) if fmt == "mxfp4" else (0, 127)
        A, Bm = codes(rng, 1, K, fmt, lo, hi), codes(rng, N, K, fmt, lo, hi)
        check_product(g.fp4_matmul(A, Bm, out_dtype=F32), A, Bm)


@pytest.mark.parametrize("ea,eb", [((0, 3), (250, 255)), ((250, 255), (0, 3)), ((0, 2), (126, 130)),
                                   ((126, 129), (0, 2)), ((127, 128), (225, 230))])
def test_one_row_of_far_scales(g, ea, eb):
    """Each scale at fp32's ends, their product inside: no step in between leaves its range."""
    rng = np.random.default_rng(3)
    A, Bm = codes(rng, 1, 320, "mxfp4", *ea), codes(rng, 140, 320, "mxfp4", *eb)
    (a, _), (b, _) = parts(A), parts(Bm)
    want, got = a @ b.T, host(g.fp4_matmul(A, Bm, out_dtype=F32))
    # as in bound(), and half of fp32's least step for each addition to a sum near it
    tol = (np.abs(a) @ np.abs(b).T) * 320 * 2.0 ** -23 + 320 * 2.0 ** -150
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_row_scaled(g, fmt):
    """Row scales: none, one for all, each its own, their product outside fp32's range."""
    rng = np.random.default_rng(5)
    A0 = g.fp4_quantize(make(rng, 1, 400).cuda().float(), fmt)
    B0 = g.fp4_quantize(make(rng, 200, 400).cuda().float(), fmt)
    one = torch.tensor([0.3], device="cuda")
    for ra in (None, one, 1e30 * one):
        for rb in (None, one.expand(200), torch.rand(400, device="cuda")[::2], 1e-30 * torch.rand(
                200, device="cuda")):
            A = Fp4Matrix(A0.data, A0.scale, ra, (1, 400), fmt)
            Bm = Fp4Matrix(B0.data, B0.scale, rb, (200, 400), fmt)
            check_product(g.fp4_matmul(A, Bm, out_dtype=F32), A, Bm)
    A = Fp4Matrix(A0.data, A0.scale, 1e30 * one, (1, 400), fmt)
    Bm = Fp4Matrix(B0.data, B0.scale, 1e30 * one.expand(200), (200, 400), fmt)
    C = g.fp4_matmul(A, Bm, out_dtype=F32)  # beyond fp32, but for sums of 0
    assert bool((torch.isinf(C) | (C == 0)).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows", [1, 20, 40, 200])
def test_rows_after_their_operands_were_written(g, rows, fmt):
    """In a chain of launches that start early: the weight quantised just before the product
    that reads it, again and again into the same memory."""
    rng = np.random.default_rng(9)
    ws = [make(rng, 600, 1100).cuda().float() for _ in range(4)]
    xs = [make(rng, rows, 1100).cuda().float() for _ in range(4)]
    want = []
    for x, w in zip(xs, ws):
        want.append(g.fp4_matmul(g.fp4_quantize(x, fmt), g.fp4_quantize(w, fmt), out_dtype=F32))
        torch.cuda.synchronize()
    x, w = xs[0].clone(), ws[0].clone()
    graph = torch.cuda.CUDAGraph()
    outs = []
    with torch.cuda.graph(graph):
        for i in range(4):
            x.copy_(xs[i])
            w.copy_(ws[i])
            outs.append(g.fp4_matmul(g.fp4_quantize(x, fmt), g.fp4_quantize(w, fmt),
                                     out_dtype=F32))
    for _ in range(10):
        for o in outs:
            o.zero_()
        graph.replay()
        assert all(torch.equal(o, v) for o, v in zip(outs, want))


def same(a, b):
    """Equal bits, of which NaN is any."""
    return a.shape == b.shape and bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("K", [1, 15, 16, 17, 33, 64, 1000, 4095, 4096, 4100, 10001, 65536, 65600])
def test_one_row_of_a_layer_is_quantising_and_product(g, K, dtype, fmt):
    """One launch, the bits of two: values of far magnitudes, zeros, non-finite ones, rows that
    do not start on 16 bytes."""
    rng = np.random.default_rng(K)
    w = g.fp4_quantize(make(rng, 300, K).cuda().float(), fmt)
    bias = torch.randn(300, device="cuda")
    buf = make(rng, 1, K + 9, 3.0).cuda().to(dtype)
    buf[0, 5] = 0
    rows = [buf[:, :K], buf[:, 1:K + 1], buf[:, 9:], torch.zeros_like(buf[:, :K]),
            buf[:, :K] * 1e-6, buf[:, :K] * 1e3]
    for bad in (float("nan"), float("inf")):
        x = buf[:, :K].clone()
        x[0, K // 2] = bad
        rows.append(x)
    for x in rows:
        for b in (None, bias):
            want = g.fp4_matmul(g.fp4_quantize(x, fmt), w, b, out_dtype=dtype)
            assert same(fp4.linear(g, x, w, b), want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_row_of_a_layer_elsewhere(g, fmt):
    """Odd widths, another result type (the C entry), row scales of the weight, empty sizes, a
    graph, another stream."""
    rng = np.random.default_rng(1)
    x = make(rng, 1, 1100).cuda().bfloat16()
    for N in (1, 31, 129, 5000):
        w = g.fp4_quantize(make(rng, N, 1100).cuda().float(), fmt)
        w = Fp4Matrix(w.data, w.scale, torch.rand(2 * N, device="cuda")[::2], w.shape, fmt)
        want = g.fp4_matmul(g.fp4_quantize(x, fmt), w, out_dtype=F32)
        y = torch.full((N + 2,), 7.0, device="cuda")
        assert B.gemm_fp4_linear_row(g.handle, N, 1100, x.data_ptr(), B.GEMM_BF16, w.desc(), None,
                                     y[1:].data_ptr(), B.GEMM_F32,
                                     torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(y[1:N + 1], want[0]) and float(y[0]) == 7 and float(y[N + 1]) == 7
    want = fp4.linear(g, x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fp4.linear(g, x, w, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    static, graph = torch.zeros_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fp4.linear(g, fp4.linear(g, static, w)[:, :1100].contiguous(), w)
    static.copy_(x)
    graph.replay()
    assert torch.equal(out, fp4.linear(g, want[:, :1100].contiguous(), w))
    bias = torch.randn(6, device="cuda")
    empty = g.fp4_quantize(torch.zeros(6, 0, device="cuda"), fmt)
    none = g.fp4_quantize(torch.zeros(0, 1100, device="cuda"), fmt)
    assert torch.equal(fp4.linear(g, torch.zeros(1, 0, device="cuda"), empty, bias)[0], bias)
    assert fp4.linear(g, x, none).shape == (1, 0)


# ------------------------------------------- splits at their ends, far scales, options --
class Options:
    """Options of a handle within a block."""

    def __init__(self, g, **forced):
        names = {"swap": B.GEMM_OPT_FORCE_SWAP_AB, "tile": B.GEMM_OPT_FORCE_TILE_N,
                 "split": B.GEMM_OPT_CLUSTER_SPLIT}
        self.g, self.forced = g, {names[k]: v for k, v in forced.items()}

    def __enter__(self):
        for o, v in self.forced.items():
            self.g.set_option(o, v)

    def __exit__(self, *_):
        for o in self.forced:
            self.g.set_option(o, -1)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("split", [2, 4, 8])
@pytest.mark.parametrize("K", [200, 257, 513, 1281, 1400, 1537, 1790, 1793, 2049, 2305])
@pytest.mark.parametrize("M,N,swap,tile", [(1, 300, 1, -1), (3, 64, 1, -1), (50, 200, 1, -1),
                                           (70, 200, 0, 64), (70, 200, 0, 128)])
def test_forced_splits_over_few_k_blocks(g, M, N, swap, tile, K, split, fmt):
    """1 to 10 k-blocks over 2, 4 and 8 CTAs: as many as CTAs, one more, uneven shares, and
    fewer, which are not split.  One row stays on the tensor cores."""
    rng = np.random.default_rng(K + split)
    A = g.fp4_quantize(make(rng, M, K).cuda().float(), fmt)
    Bm = g.fp4_quantize(make(rng, N, K).cuda().float(), fmt)
    with Options(g, swap=swap, tile=tile, split=split):
        for _ in range(2):
            check_product(g.fp4_matmul(A, Bm, out_dtype=F32), A, Bm)
    g.status()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("K", [1536, 1537, 1792, 1793, 2048, 2049, 2304, 2305, 2560, 2561])
@pytest.mark.parametrize("M,N", [(3, 64), (20, 1000), (70, 200), (128, 1024)])
def test_splits_around_their_rule(g, M, N, K, fmt):
    """No option set: 6 to 11 k-blocks, from which on a split pays, on both sides."""
    rng = np.random.default_rng(K)
    A = g.fp4_quantize(make(rng, M, K).cuda().float(), fmt)
    Bm = g.fp4_quantize(make(rng, N, K).cuda().float(), fmt)
    for _ in range(2):
        check_product(g.fp4_matmul(A, Bm, out_dtype=F32), A, Bm)
    g.status()


@pytest.mark.parametrize("ea,eb", [((0, 3), (250, 255)), ((250, 255), (0, 3)), ((0, 2), (126, 130)),
                                   ((126, 129), (0, 2)), ((127, 128), (225, 230)),
                                   ((60, 70), (180, 190))])
@pytest.mark.parametrize("M,forced", [(1, {}), (1, dict(swap=1)), (2, {}), (33, {}), (40, {}),
                                      (40, dict(swap=1, split=2)), (300, {}), (300, dict(tile=64)),
                                      (300, dict(tile=256)), (70, dict(split=2))])
def test_products_of_far_scales(g, M, forced, ea, eb):
    """mxfp4 scales at fp32's ends, their product inside, on the tensor cores too."""
    rng = np.random.default_rng(3)
    A, Bm = codes(rng, M, 320, "mxfp4", *ea), codes(rng, 140, 320, "mxfp4", *eb)
    (a, _), (b, _) = parts(A), parts(Bm)
    want = a @ b.T
    with Options(g, **forced):
        got = host(g.fp4_matmul(A, Bm, out_dtype=F32))
    # as for one row: truncating additions, and half of fp32's least step for each
    tol = (np.abs(a) @ np.abs(b).T) * 320 * 2.0 ** -23 + 320 * 2.0 ** -150
    assert (np.abs(got - want) <= tol).all()
    g.status()


def test_one_row_and_two_agree_on_far_scales(g):
    """The same row alone (CUDA cores) and twice (tensor cores): each within its bound."""
    rng = np.random.default_rng(4)
    for ea, eb in (((0, 3), (250, 255)), ((126, 129), (0, 2)), ((127, 128), (225, 230))):
        two, Bm = codes(rng, 2, 320, "mxfp4", *ea), codes(rng, 140, 320, "mxfp4", *eb)
        data = two.data[:1].expand(2, 160).contiguous()
        byte = two.block_scales()[:1].expand(2, 10).contiguous()
        two = Fp4Matrix.from_parts(data, byte, None, 320, "mxfp4")
        one = Fp4Matrix.from_parts(data[:1], byte[:1], None, 320, "mxfp4")
        (a, _), (b, _) = parts(one), parts(Bm)
        tol = 2 * ((np.abs(a) @ np.abs(b).T) * 320 * 2.0 ** -23 + 320 * 2.0 ** -150)
        y1, y2 = (host(g.fp4_matmul(m, Bm, out_dtype=F32)) for m in (one, two))
        assert np.array_equal(y2[0], y2[1]) and (np.abs(y1 - y2[:1]) <= tol).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("forced", [{}, dict(swap=1), dict(swap=0), dict(tile=64), dict(tile=128),
                                    dict(split=4), dict(swap=1, split=0)])
def test_one_row_of_a_layer_follows_the_options(g, forced, dtype, fmt):
    """The layer's bits are those of the two calls on the same handle, whatever is forced."""
    rng = np.random.default_rng(8)
    x = make(rng, 1, 2500).cuda().to(dtype)
    w = g.fp4_quantize(make(rng, 300, 2500).cuda().float(), fmt)
    bias = torch.randn(300, device="cuda")
    with Options(g, **forced):
        assert B.gemm_fp4_one_row(g.handle, 300, 2500) == (not forced)
        for b in (None, bias):
            want = g.fp4_matmul(g.fp4_quantize(x, fmt), w, b, out_dtype=dtype)
            assert torch.equal(fp4.linear(g, x, w, b), want)
            check_product(want, g.fp4_quantize(x, fmt), w, b)
    g.status()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("N", [24576, 32767, 32768, 32769, 65536])
def test_one_row_on_both_sides_of_its_rule(g, N, fmt):
    """Up to 2^15 rows of B on the CUDA cores, in several rounds of CTAs; more on the tensor
    cores; a layer's row the same bits as two calls on both."""
    K = 150
    assert B.gemm_fp4_one_row(g.handle, N, K) == (N < 32768)
    rng = np.random.default_rng(N)
    w = g.fp4_quantize(make(rng, N, K).cuda().float(), fmt)
    x = make(rng, 1, K).cuda().bfloat16()
    bias = torch.randn(N, device="cuda")
    for b in (None, bias):
        q = g.fp4_quantize(x, fmt)
        C = g.fp4_matmul(q, w, b, out_dtype=F32)
        check_product(C, q, w, b)
        assert torch.equal(fp4.linear(g, x, w, b), g.fp4_matmul(q, w, b, out_dtype=BF16))
    y = torch.empty(1, N, device="cuda")  # the row's kernel itself
    assert B.gemm_fp4_linear_row(g.handle, N, K, x.data_ptr(), B.GEMM_BF16, w.desc(),
                                 bias.data_ptr(), y.data_ptr(), B.GEMM_F32,
                                 torch.cuda.current_stream().cuda_stream) == 0
    check_product(y, q, w, bias)
    g.status()
