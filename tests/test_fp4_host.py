"""The 4-bit operators' and the orthogonalising call's host side, without a GPU: argument
checks of the C-ABI and of the Python calls, sizes and layouts, and the oracle itself."""
import ctypes

import numpy as np
import pytest
import torch

import fp4_reference as R
from dense_gemm_tmem_gb300 import binding as B
from dense_gemm_tmem_gb300 import fp4
from dense_gemm_tmem_gb300.fp4 import Fp4Matrix
from dense_gemm_tmem_gb300.gemm import Gemm, _coefficients

ERR, UNSUPPORTED = B.GEMM_ERR_INVALID_ARG, B.GEMM_ERR_UNSUPPORTED


def matrix(fmt=B.GEMM_MXFP4, ld=64, data=16, scale=16, rows=None, stride=1):
    return B.gemm_fp4_matrix_t(data, ld, scale, rows, stride, fmt, 0)


def test_structs_match_the_header():
    assert ctypes.sizeof(B.gemm_fp4_matrix_t) == 48
    assert ctypes.sizeof(B.gemm_orthogonalize_t) == 24 + 8 + 16 + 48


@pytest.fixture()
def handle():
    """Memory in a handle's place: calls that are refused look at nothing in it."""
    buf = ctypes.create_string_buffer(1 << 20)
    return ctypes.addressof(buf), buf


def test_quantise_refusals(handle):
    h, _ = handle
    def call(rows=4, cols=64, src=16, ld=64, dtype=B.GEMM_F32, m=None, handle=h):
        return B.gemm_fp4_quantize(handle, rows, cols, src, ld, dtype, m or matrix(), None)
    nv = dict(fmt=B.GEMM_NVFP4)
    assert call(handle=None) == ERR
    assert call(rows=-1) == ERR and call(cols=-1) == ERR and call(ld=63) == ERR
    assert call(dtype=3) == ERR and call(dtype=-1) == ERR and call(src=None) == ERR
    assert call(m=matrix(fmt=2)) == ERR and call(m=matrix(ld=16)) == ERR
    assert call(m=matrix(data=None)) == ERR and call(m=matrix(scale=None)) == ERR
    assert call(m=matrix(rows=16)) == ERR                  # mxfp4 has no row scale
    assert call(m=matrix(**nv)) == ERR                     # nvfp4 needs one
    assert call(m=matrix(rows=16, stride=0, **nv)) == ERR  # of its own for each row
    assert call(m=matrix(ld=65)) == UNSUPPORTED
    assert call(m=matrix(data=24)) == UNSUPPORTED and call(m=matrix(scale=17)) == UNSUPPORTED
    assert call(rows=2 ** 31) == UNSUPPORTED
    assert call(cols=2 ** 31, ld=2 ** 31, m=matrix(ld=2 ** 31)) == UNSUPPORTED
    assert call(rows=0) == 0 and call(cols=0, ld=0) == 0   # nothing to do


def test_read_back_and_product_refusals(handle):
    h, _ = handle
    m = matrix()
    assert B.gemm_fp4_dequantize(None, 4, 64, m, 16, 64, B.GEMM_F32, None) == ERR
    assert B.gemm_fp4_dequantize(h, 4, 64, m, 16, 63, B.GEMM_F32, None) == ERR
    assert B.gemm_fp4_dequantize(h, 4, 64, m, None, 64, B.GEMM_F32, None) == ERR
    assert B.gemm_fp4_dequantize(h, 4, 64, matrix(ld=72), 16, 64, B.GEMM_F32, None) == UNSUPPORTED
    assert B.gemm_fp4_dequantize(h, 0, 64, m, None, 64, B.GEMM_F32, None) == 0

    def run(M=4, N=8, K=64, A=m, Bm=m, C=16, ldc=8, dtype=B.GEMM_F32, handle=h):
        return B.gemm_fp4_run(handle, M, N, K, A, Bm, None, C, ldc, dtype, None)
    assert run(handle=None) == ERR
    assert run(M=-1) == ERR and run(N=-1) == ERR and run(K=-1) == ERR
    assert run(ldc=7) == ERR and run(C=None) == ERR and run(dtype=9) == ERR
    assert run(Bm=matrix(fmt=B.GEMM_NVFP4)) == ERR
    assert run(A=matrix(ld=16)) == ERR and run(Bm=matrix(data=None)) == ERR
    assert run(A=matrix(ld=40)) == UNSUPPORTED and run(Bm=matrix(scale=8)) == UNSUPPORTED
    assert run(M=2 ** 31) == UNSUPPORTED
    assert run(M=0) == 0 and run(N=0, ldc=0) == 0


def test_row_of_a_layer_refusals(handle):
    h, _ = handle
    m = matrix()
    def row(N=8, K=64, x=16, dtype=B.GEMM_BF16, W=m, bias=None, y=16, out=B.GEMM_BF16, handle=h):
        return B.gemm_fp4_linear_row(handle, N, K, x, dtype, W, bias, y, out, None)
    assert row(handle=None) == ERR and row(N=-1) == ERR and row(K=-1) == ERR
    assert row(dtype=9) == ERR and row(out=-1) == ERR and row(x=None) == ERR and row(y=None) == ERR
    assert row(W=matrix(ld=16)) == ERR and row(W=matrix(data=None)) == ERR
    assert row(W=matrix(fmt=2)) == ERR
    assert row(x=17) == UNSUPPORTED and row(y=18, out=B.GEMM_F32) == UNSUPPORTED
    assert row(bias=18) == UNSUPPORTED and row(W=matrix(ld=40)) == UNSUPPORTED
    assert row(K=65537, W=matrix(ld=1 << 16)) == UNSUPPORTED
    assert row(N=2 ** 31) == UNSUPPORTED and row(N=0, x=None, y=None) == 0


def test_one_row_asks_for_a_handle_and_sizes(handle):
    h, _ = handle
    assert B.gemm_fp4_one_row(None, 8, 64) == 0
    assert B.gemm_fp4_one_row(h, -1, 64) == 0 and B.gemm_fp4_one_row(h, 8, -1) == 0


def ortho(**kw):
    abc = (ctypes.c_float * 192)(*([3.4445, -4.7750, 2.0315] * 64))
    p = dict(batch=1, rows=64, cols=32, steps=5, dtype=B.GEMM_F32,
             coefficients=ctypes.addressof(abc), eps=1e-7, g=256, ld_g=32, stride_g=0, out=256,
             ld_out=32, stride_out=0)
    p.update(kw)
    q = B.gemm_orthogonalize_t(**p)
    q.keep = abc
    return q


def test_orthogonalize_refusals(handle):
    h, _ = handle
    def call(ws=256, size=1 << 40, handle=h, **kw):
        return B.gemm_orthogonalize(handle, ortho(**kw), ws, size, None)
    assert call(handle=None) == ERR
    for bad in (dict(batch=-1), dict(rows=-1), dict(cols=-1), dict(steps=0), dict(steps=65),
                dict(dtype=3), dict(coefficients=None), dict(eps=0.0), dict(eps=float("nan")),
                dict(eps=2.0 ** 101), dict(ld_g=31), dict(ld_out=31), dict(g=None),
                dict(out=None), dict(ws=None), dict(ws=128), dict(size=1000),
                dict(batch=2, stride_out=1000), dict(batch=2, stride_g=-1, stride_out=2048)):
        assert call(**bad) == ERR, bad
    assert call(rows=1 << 20) == UNSUPPORTED and call(batch=1 << 16) == UNSUPPORTED
    for empty in (dict(batch=0), dict(rows=0), dict(cols=0)):
        assert call(g=None, out=None, ws=None, **empty) == 0
    for abc in ([float("inf"), 0, 0], [float("nan"), 0, 0], [1e5, 0, 0], [0, 0, 2e4],
                [3, 1e9, -1e9]):
        c = (ctypes.c_float * 15)(*(abc * 5))
        assert call(coefficients=ctypes.addressof(c)) == ERR, abc


def test_addresses_inside_an_element_are_refused(handle):
    h, _ = handle
    m, nv = matrix(), matrix(rows=18, fmt=B.GEMM_NVFP4)
    for dtype, at in ((B.GEMM_F32, 18), (B.GEMM_F16, 17), (B.GEMM_BF16, 33)):
        assert B.gemm_fp4_quantize(h, 4, 64, at, 64, dtype, m, None) == UNSUPPORTED
        assert B.gemm_fp4_dequantize(h, 4, 64, m, at, 64, dtype, None) == UNSUPPORTED
        assert B.gemm_fp4_run(h, 4, 8, 64, m, m, None, at, 8, dtype, None) == UNSUPPORTED
        assert B.gemm_orthogonalize(h, ortho(g=at, dtype=dtype), 256, 1 << 40, None) == UNSUPPORTED
    assert B.gemm_fp4_run(h, 4, 8, 64, m, m, 18, 16, 8, B.GEMM_F32, None) == UNSUPPORTED
    assert B.gemm_fp4_quantize(h, 4, 64, 16, 64, B.GEMM_F32, nv, None) == UNSUPPORTED
    assert B.gemm_orthogonalize(h, ortho(out=257), 256, 1 << 40, None) == UNSUPPORTED


def test_coefficients_that_lose_the_iterate_are_refused(handle):
    """16-bit copies of an iterate far below 1 have scales that fp32 does not hold."""
    h, _ = handle
    def call(*abc):
        c = (ctypes.c_float * (3 * len(abc)))(*(v for step in abc for v in step))
        p = ortho(steps=len(abc), coefficients=ctypes.addressof(c), g=None)
        return B.gemm_orthogonalize(h, p, None, 0, None), \
            B.gemm_orthogonalize(h, ortho(steps=len(abc), coefficients=ctypes.addressof(c), rows=0),
                                 None, 0, None)
    assert call((1e-15, 0, 0), (0, 1e38, 0)) == (ERR, ERR)
    assert call((2.0 ** -21, 0, 0), (1, 0, 0)) == (ERR, ERR)
    # accepted, so that only the missing pointers are left: small but held, zero, the last step
    for ok in (((2.0 ** -20, 0, 0), (1, 0, 0)), ((0, 0, 0), (1, 0, 0)), ((1, 0, 0), (1e-15, 0, 0))):
        assert call(*ok) == (ERR, 0)


def test_orthogonalize_workspace(handle):
    h, _ = handle
    assert B.gemm_orthogonalize_workspace(None, ortho()) == (ERR, 0)
    assert B.gemm_orthogonalize_workspace(h, ortho(steps=0)) == (ERR, 0)
    assert B.gemm_orthogonalize_workspace(h, ortho(cols=1 << 20)) == (UNSUPPORTED, 0)
    rc, small = B.gemm_orthogonalize_workspace(h, ortho(rows=1000, cols=1000, ld_g=1000))
    # the iterate in fp32 and twice in 16 bits, A and B, rows padded to 64
    assert rc == 0 and 1000 * 1024 * 12 <= small <= 1000 * 1024 * 12 + (1 << 20)
    assert B.gemm_orthogonalize_workspace(h, ortho(rows=1000, cols=1000, batch=3))[1] > 2.5 * small


def test_scale_bytes():
    for rows in (0, 1, 127, 128, 129, 1000):
        for cols in (0, 1, 16, 33, 64, 65, 128, 4100):
            for fmt, code in fp4.FORMATS.items():
                blocks = -(-cols // R.BLOCK[fmt])
                want = -(-rows // 128) * -(-blocks // 4) * 512
                assert fp4.scale_bytes(rows, cols, fmt) == want
                assert B.gemm_fp4_scale_bytes(rows, cols, code) == want
    assert B.gemm_fp4_scale_bytes(-1, 4, 0) == ERR and B.gemm_fp4_scale_bytes(4, 4, 2) == ERR


@pytest.mark.parametrize("rows,blocks", [(1, 1), (33, 4), (128, 5), (300, 13)])
def test_scales_are_packed_where_the_header_says(rows, blocks):
    rng = np.random.default_rng(rows)
    s = torch.from_numpy(rng.integers(1, 256, (rows, blocks)).astype(np.uint8))
    p = fp4.pack_scales(s)
    r, b = np.arange(rows)[:, None], np.arange(blocks)[None, :]
    want = np.zeros(p.numel(), np.uint8)
    want[R.place(r, b, blocks)] = s.numpy()
    assert np.array_equal(p.numpy(), want)
    assert torch.equal(fp4.unpack_scales(p, rows, blocks), s)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 45), (130, 64)])
def test_from_parts(fmt, rows, cols):
    rng = np.random.default_rng(cols)
    code, byte, rs = R.quantize(rng.standard_normal((rows, cols)), fmt)
    rs = None if rs is None else torch.from_numpy(rs).float()
    m = Fp4Matrix.from_parts(torch.from_numpy(R.pack(code)), torch.from_numpy(byte), rs, cols, fmt)
    got_code, got_byte = R.stored(m)
    assert np.array_equal(got_code, code) and np.array_equal(got_byte, byte)
    assert m.data.stride(0) % 16 == 0 or rows == 1
    assert torch.equal(m.block_scales(), torch.from_numpy(byte))
    one = Fp4Matrix.from_parts(m.data, torch.from_numpy(byte), torch.tensor(0.5), cols, fmt)
    assert one.row_scale.shape == (rows,) and one.row_scale.stride(0) == 0 or rows == 1
    if cols % 2:  # the odd column's partner is cleared
        dirty = m.data.clone() | torch.tensor([0] * (m.data.shape[1] - 1) + [0xf0],
                                              dtype=torch.uint8)
        again = Fp4Matrix.from_parts(dirty, torch.from_numpy(byte), rs, cols, fmt)
        assert torch.equal(again.data, m.data)


@pytest.mark.parametrize("loaded", [False, True])
def test_matrix_refusals(monkeypatch, loaded):
    """The same refusals with the extension's checks and without the extension."""
    monkeypatch.setattr(B, "_native", B.native() if loaded else None)
    data = torch.zeros(4, 32, dtype=torch.uint8)
    scale = torch.zeros(512, dtype=torch.uint8)
    rs = torch.ones(4)
    Fp4Matrix(data, scale, None, (4, 64), "mxfp4")
    Fp4Matrix(data, scale, rs, (4, 64), "nvfp4")
    for args, error in (((data.float(), scale, None, (4, 64), "mxfp4"), TypeError),
                        ((data, scale.float(), None, (4, 64), "mxfp4"), TypeError),
                        ((data, scale, rs.double(), (4, 64), "nvfp4"), TypeError),
                        ((data, scale, rs[:3], (4, 64), "nvfp4"), ValueError),
                        ((data, scale, None, (4, 66), "mxfp4"), ValueError),
                        ((data, scale, None, (5, 64), "mxfp4"), ValueError),
                        ((data, scale[:511], None, (4, 64), "mxfp4"), ValueError),
                        ((data, scale.view(2, 256), None, (4, 64), "mxfp4"), ValueError),
                        ((data.t(), scale, None, (32, 8), "mxfp4"), ValueError),
                        ((data, scale, None, (4, 64), "fp4"), ValueError)):
        with pytest.raises(error):
            Fp4Matrix(*args)
    for args in ((data, torch.zeros(4, 3, dtype=torch.uint8), None, 64, "nvfp4"),
                 (data, torch.zeros(4, 4, dtype=torch.uint8), None, 66, "nvfp4")):
        with pytest.raises(ValueError):
            Fp4Matrix.from_parts(*args)


def no_handle():
    """A Gemm without a device, for the checks that come before it is used."""
    g = object.__new__(Gemm)
    g.device, g.handle, g._native = torch.device("cuda", 0), 0, None
    return g


def test_python_calls_refuse_before_the_gpu():
    g = no_handle()
    mx = Fp4Matrix(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8),
                   None, (4, 64), "mxfp4")
    nv = Fp4Matrix(mx.data, mx.scale, torch.ones(4), (4, 64), "nvfp4")
    short = Fp4Matrix(mx.data[:, :16], mx.scale, None, (4, 32), "mxfp4")
    with pytest.raises(ValueError, match="mxfp4"):
        g.fp4_quantize(torch.zeros(4, 4), "e2m1")
    for a, b in ((mx, nv), (mx, short)):
        with pytest.raises(ValueError):
            g.fp4_matmul(a, b)
        with pytest.raises(ValueError):
            g.fp4_run(a, b, torch.zeros(4, 4))
    with pytest.raises(TypeError):
        g.fp4_matmul(mx, mx, out_dtype=torch.float64)
    with pytest.raises(TypeError):
        g.fp4_dequantize(mx, torch.float64)
    with pytest.raises(ValueError, match="steps"):
        g.orthogonalize(torch.zeros(4, 4), 0)
    for abc in ((1, 2), [(1, 2, 3)], [(1, 2, 3)] * 4, [(1, 2)] * 5, ()):
        with pytest.raises(ValueError, match="coefficients"):
            g.orthogonalize(torch.zeros(4, 4), 5, abc)
    g.handle = None


def test_extension_refuses_host_tensors_and_replaced_ones():
    n = B.native()
    x = torch.zeros(3, 64)
    data = torch.zeros(3, 32, dtype=torch.uint8)
    scale, rs = torch.zeros(512, dtype=torch.uint8), torch.ones(3)

    def product(call, data=data, scale=scale, rs=rs, cols=64, kind=1, last=0):
        ok = (torch.zeros(3, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), None)
        return getattr(n, call)(1, 0, data, scale, rs, *ok, cols, kind, None, last, 0)

    for call in (lambda: n.quantize4(1, 0, x, 0, 0),
                 lambda: n.dequantize4(1, 0, data, scale, rs, 64, 1, 0, 0),
                 lambda: product("matmul4"), lambda: product("run4", last=torch.zeros(3, 3)),
                 lambda: n.linear4(1, 0, x, data, scale, rs, 64, 1, None, 0),
                 lambda: n.orthogonalize(1, 0, x, b"\0" * 12, 1e-7, 0)):
        with pytest.raises(ValueError, match="device"):
            call()
    for change, error in ((dict(data=data.float()), TypeError), (dict(data=data[0]), ValueError),
                          (dict(data=data[:, :31]), ValueError), (dict(cols=-2), ValueError),
                          (dict(scale=scale[:100]), ValueError), (dict(scale=None), TypeError),
                          (dict(scale=scale.float()), TypeError), (dict(kind=2), ValueError)):
        with pytest.raises(error):
            product("matmul4", **change)
    for call in (lambda: n.quantize4(1, 0, x.double(), 0, 0), lambda: n.quantize4(1, 0),
                 lambda: n.quantize4(1, 0, "x", 0, 0), lambda: n.matmul4(1),
                 lambda: n.orthogonalize(1, 0, x.double(), b"\0" * 12, 1e-7, 0)):
        with pytest.raises(TypeError):
            call()


def test_coefficients():
    one = np.frombuffer(_coefficients((1.0, 2.0, 3.0), 2), np.float32)
    assert np.array_equal(one, [1, 2, 3, 1, 2, 3])
    each = np.frombuffer(_coefficients([(1, 2, 3), (4, 5, 6)], 2), np.float32)
    assert np.array_equal(each, [1, 2, 3, 4, 5, 6])


@pytest.mark.parametrize("steps", [1, 2, 3, 5])
def test_one_triple_in_any_numbers(steps):
    """A triple for every step, as a tensor, an array or numbers without dimensions, also where
    there are three steps."""
    want = np.tile(np.array([1, 2, 3], np.float32), steps)
    for abc in ((1, 2, 3), [1.0, 2.0, 3.0], torch.tensor([1.0, 2.0, 3.0]), np.arange(1.0, 4.0),
                tuple(torch.tensor([1.0, 2.0, 3.0])), [np.array(v) for v in (1, 2, 3)],
                (v for v in (1, 2, 3))):
        assert np.array_equal(np.frombuffer(_coefficients(abc, steps), np.float32), want)
    for bad in ((1, 2), (1, 2, 3, 4), torch.ones(4), torch.ones(steps + 1, 3), torch.ones(steps, 2)):
        with pytest.raises(ValueError, match="coefficients"):
            _coefficients(bad, steps)


def test_coefficients_changed_in_place():
    """What a caller's object holds now counts, not what it held in an earlier call."""
    first, then = (3.4445, -4.7750, 2.0315), (1.875, -1.25, 0.375)
    made = (lambda v: torch.tensor([v] * 3), lambda v: tuple(torch.tensor(v) for _ in range(3)),
            lambda v: np.array([v] * 3, np.float32), lambda v: [list(v) for _ in range(3)],
            lambda v: tuple([x for x in v] for _ in range(3)),
            lambda v: tuple(tuple(torch.tensor(x) for x in v) for _ in range(3)))
    for make in made:
        abc = make(first)
        want = np.tile(np.array(first, np.float32), 3)
        assert np.array_equal(np.frombuffer(_coefficients(abc, 3), np.float32), want)
        for row in abc:
            for i, v in enumerate(then):
                if isinstance(row, tuple):
                    row[i].fill_(v)
                else:
                    row[i] = v
        want = np.tile(np.array(then, np.float32), 3)
        assert np.array_equal(np.frombuffer(_coefficients(abc, 3), np.float32), want)
    one = [1.0, 2.0, 3.0]
    _coefficients(one, 2)
    one[0] = 5.0
    assert np.array_equal(np.frombuffer(_coefficients(one, 2), np.float32), [5, 2, 3] * 2)


def test_reference_rounds_to_the_nearest_value():
    """The oracle's e2m1 and e4m3 against a search of their values."""
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-8, 8, 4000), np.arange(-32, 33) / 4.0])
    got = R.E2M1[R.round_e2m1(v) & 7] * np.where(R.round_e2m1(v) & 8, -1, 1)
    far = np.abs(v[:, None] - np.concatenate([R.E2M1, -R.E2M1])[None, :]).min(1)
    assert np.array_equal(np.abs(v - got), far)
    assert [int(c) for c in R.round_e2m1(np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 9]))] == [
        0, 2, 2, 4, 4, 6, 6, 7]
    w = np.concatenate([rng.uniform(0, 448, 2000), rng.uniform(0, 0.1, 2000)])
    w = w.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(w).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.to_e4m3(w), want)
    b = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    assert np.array_equal(R.e4m3(b.numpy()), b.view(torch.float8_e4m3fn).double().numpy(),
                          equal_nan=True)
