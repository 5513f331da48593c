"""The 8-bit operators' host side, without a GPU: argument checks of the C-ABI
and of the Python calls, sizes and layouts."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_reference as R
from dense_gemm_tmem_gb300 import binding as B
from dense_gemm_tmem_gb300.fp8 import Fp8Matrix, scale_shape


@pytest.fixture(scope="module")
def lib():
    return B.load()


def matrix(blocks=B.GEMM_FP8_ROW, ld=128, data=16, scale=16):
    return B.gemm_fp8_matrix_t(data, ld, scale, 1, 1, blocks, 0)


def test_null_handle_is_refused(lib):
    m = matrix()
    assert B.gemm_fp8_quantize(None, 1, 1, 16, 1, B.GEMM_F32, m, None, None) == -1
    assert B.gemm_fp8_run(None, 1, 1, 1, m, m, None, 16, 1, 0, 1, B.GEMM_F32, None) == -1
    layer = B.gemm_moe_fp8_t(tokens=1, hidden=64, inner=64, experts=4, top_k=1)
    assert B.gemm_moe_fp8_workspace(None, layer) == (B.GEMM_ERR_INVALID_ARG, 0)
    assert B.gemm_moe_fp8(None, layer, None, 0, None) == B.GEMM_ERR_INVALID_ARG


def test_structs_match_the_header(lib):
    """Sizes of the C structs (all 8-byte fields but pairs of int32)."""
    assert ctypes.sizeof(B.gemm_fp8_matrix_t) == 48
    assert ctypes.sizeof(B.gemm_fp8_experts_t) == 56
    assert ctypes.sizeof(B.gemm_moe_fp8_t) == 32 + 16 + 32 + 3 * 56 + 32


@pytest.mark.parametrize("rows,cols", [(1, 1), (128, 128), (129, 257), (5, 4096)])
def test_scale_shapes(rows, cols):
    rb, cb = -(-rows // 128), -(-cols // 128)
    assert scale_shape(rows, cols, "row") == (rows, cb)
    assert scale_shape(rows, cols, "col") == (rb, cols)
    assert scale_shape(rows, cols, "tile") == (rb, cb)
    with pytest.raises(ValueError):
        scale_shape(rows, cols, "line")


@pytest.mark.parametrize("blocks", ["row", "col", "tile"])
def test_empty_layout_and_values(blocks):
    m = Fp8Matrix.empty(130, 300, blocks, "cpu")
    assert m.data.shape == (130, 300) and m.data.stride() == (304, 1)
    assert m.scale.shape == scale_shape(130, 300, blocks)
    if blocks == "row":
        assert m.scale.stride()[0] == 1
    rng = np.random.default_rng(0)
    q, s = R.quantize(rng.standard_normal((130, 300)), blocks)
    m.data.copy_(torch.from_numpy(q).float().to(torch.float8_e4m3fn))
    m.scale.copy_(torch.from_numpy(s))
    assert np.array_equal(m.dequantize().double().numpy(),
                          (q.astype(np.float32) * R.spread(s, 130, 300, blocks)).astype(np.float64))


def test_matrix_refusals():
    data = torch.zeros(4, 256, dtype=torch.uint8)
    scale = torch.zeros(4, 2)
    Fp8Matrix(data, scale, "row")
    for args, error in (((data.float(), scale, "row"), TypeError),
                        ((data, scale.double(), "row"), TypeError),
                        ((data, scale, "rows"), ValueError),
                        ((data, scale[:, :1], "row"), ValueError),
                        ((data.t(), scale, "row"), ValueError),
                        ((data[0], scale, "row"), ValueError),
                        ((data[None], scale[None], "row"), ValueError)):
        with pytest.raises(error):
            Fp8Matrix(*args)


def test_calls_refuse_host_tensors():
    n = B.native()
    x = torch.zeros(3, 64)
    m = Fp8Matrix.empty(3, 64, "row", "cpu")
    w = Fp8Matrix.empty(8, 64, "tile", "cpu")
    for call in (lambda: n.quantize(1, 0, x, 0, -1, 0),
                 lambda: n.matmul(1, 0, m.data, m.scale, 0, w.data, w.scale, 2, None, 0, 1, 0, 0),
                 lambda: n.moe(1, 0, x.half(), x.half(), *([w.data, w.scale] * 3), 1, 1, 0)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: n.quantize(1, 0, x.double(), 0, -1, 0), lambda: n.quantize(1, 0),
                 lambda: n.quantize(1, 0, "x", 0, -1, 0),
                 lambda: n.moe(1, 0, x, x, *([w.data, w.scale] * 3), 1, 1, 0)):
        with pytest.raises(TypeError):
            call()


def test_reference_rounds_like_torch():
    """The oracle's e4m3 rounding against torch's conversion, ties included."""
    grid = np.arange(0, 256, dtype=np.uint8)
    v = torch.from_numpy(grid).view(torch.float8_e4m3fn).double().numpy()
    v = np.sort(np.unique(v[np.isfinite(v)]))
    mids = (v[1:] + v[:-1]) / 2
    near = np.concatenate([v, mids, np.nextafter(mids, 1e9), np.nextafter(mids, -1e9)])
    near = near.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(near).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.round_e4m3(near), want)


def test_reference_layer_against_a_plain_loop():
    rng = np.random.default_rng(3)
    T, H, I, E, k = 3, 40, 24, 5, 2
    x, r = rng.standard_normal((T, H)), rng.standard_normal((E, H))
    w1, w3, w2 = (rng.standard_normal(s) for s in ((E, I, H), (E, I, H), (E, H, I)))
    ids = np.argsort(-(x @ r.T), 1, kind="stable")[:, :k]
    out, _, gates, _ = R.moe(x, r, w1, w3, w2, ids, True)
    for t in range(T):
        l = x[t] @ r.T
        xq = R.values(*R.quantize(x[t:t + 1], "row"), "row")[0]
        want, norm = 0.0, sum(np.exp(l[e]) for e in ids[t])
        for j, e in enumerate(ids[t]):
            assert abs(gates[t, j] - np.exp(l[e]) / norm) < 1e-12
            a = w1[e] @ xq
            h = a / (1 + np.exp(-a)) * (w3[e] @ xq)
            h = R.values(*R.quantize(h[None], "row"), "row")[0]
            want = want + np.exp(l[e]) / norm * (w2[e] @ h)
        assert np.allclose(out[t], want, rtol=1e-12, atol=1e-12)
