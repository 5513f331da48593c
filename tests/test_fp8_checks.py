"""The extension looks at a block-scaled matrix's tensors on every call, whatever
became of the Fp8Matrix since it was made: without a GPU, by what it refuses before
it asks for one."""
import pytest
import torch

from dense_gemm_tmem_gb300 import binding as B
from dense_gemm_tmem_gb300.fp8 import Fp8Matrix


def product(call, m, w, last):
    return getattr(B.native(), call)(1, 0, m.data, m.scale, m.kind, w.data, w.scale, w.kind, None,
                                     0, 1, last, 0)


@pytest.mark.parametrize("call", ["matmul", "run"])
@pytest.mark.parametrize("blocks", ["row", "tile"])
def test_replaced_tensors_of_a_product(call, blocks):
    last = 0 if call == "matmul" else torch.zeros(200, 130)

    def matrices():
        return Fp8Matrix.empty(200, 300, blocks, "cpu"), Fp8Matrix.empty(130, 300, "tile", "cpu")

    m, w = matrices()
    with pytest.raises(ValueError, match="device"):
        product(call, m, w, last)  # as it should be, but for the device
    for which in (0, 1):
        for change, error, says in (
                (lambda t: setattr(t, "scale", t.scale.double()), TypeError, "float32"),
                (lambda t: setattr(t, "scale", t.scale[:, :1]), ValueError, "shape"),
                (lambda t: setattr(t, "scale", t.scale[:1]), ValueError, "shape"),
                (lambda t: setattr(t, "scale", t.scale.flatten()), ValueError, "2-D"),
                (lambda t: setattr(t, "data", t.data.float()), TypeError, "float8"),
                (lambda t: setattr(t, "data", t.data[:100]), ValueError, "shape"),
                (lambda t: setattr(t, "kind", B.GEMM_FP8_COL), ValueError, "shape"),
                (lambda t: setattr(t, "kind", 3), ValueError, "blocks")):
            ms = matrices()
            change(ms[which])
            with pytest.raises(error, match=says):
                product(call, *ms, last)


def test_replaced_tensors_of_an_expert_layer():
    E, H, I = 3, 300, 140

    def weights():
        def one(rows, cols):
            data = torch.zeros(E, rows, -(-cols // 16) * 16, dtype=torch.uint8)[:, :, :cols]
            return Fp8Matrix(data, torch.ones(E, -(-rows // 128), -(-cols // 128)), "tile")
        return one(I, H), one(I, H), one(H, I)

    def moe(ws):
        x = torch.zeros(2, H, dtype=torch.float16)
        return B.native().moe(1, 0, x, torch.zeros(E, H, dtype=torch.float16),
                              *(t for w in ws for t in (w.data, w.scale)), 1, 1, 0)

    with pytest.raises(ValueError, match="device"):
        moe(weights())
    for which in range(3):
        for change, error, says in (
                (lambda t: setattr(t, "scale", t.scale.half()), TypeError, "float32"),
                (lambda t: setattr(t, "scale", t.scale[:2]), ValueError, "per expert"),
                (lambda t: setattr(t, "scale", t.scale[:, :1]), ValueError, "shape"),
                (lambda t: setattr(t, "scale", t.scale[..., :1]), ValueError, "shape"),
                (lambda t: setattr(t, "data", t.data.to(torch.int16)), TypeError, "float8"),
                (lambda t: setattr(t, "data", t.data[..., :8]), ValueError, "shape"),
                (lambda t: setattr(t, "data", t.data.transpose(1, 2).contiguous()
                                   .transpose(1, 2)), ValueError, "contiguous")):
            ws = weights()
            change(ws[which])
            with pytest.raises(error, match=says):
                moe(ws)
