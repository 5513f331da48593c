"""What the 8-bit operators' Python calls hold, keep alive and check, on the GPU."""
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
    h = Gemm(torch.device("cuda", 0))
    yield h
    h.close()


def test_row_and_column_copies_do_not_hold_each_other(g):
    x = torch.randn(1024, 2048, device="cuda").bfloat16()
    row, col = g.fp8_quantize(x, "row+col")
    own = 1024 * 2048 + 4 * 1024 * 16
    for m in (row, col):
        assert m.data.untyped_storage().data_ptr() == m.scale.untyped_storage().data_ptr()
        assert m.data.untyped_storage().nbytes() <= own + 512
    assert row.data.untyped_storage().data_ptr() != col.data.untyped_storage().data_ptr()
    before = torch.cuda.memory_allocated()
    del row, m
    assert before - torch.cuda.memory_allocated() >= own
