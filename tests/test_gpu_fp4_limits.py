"""The 4-bit product under wait limits short enough to run out anywhere in a launch: it
ends, gemm_status reports it or the result is right, and the next call is right."""
import pytest
import torch

from dense_gemm_tmem_gb300 import binding as B
from dense_gemm_tmem_gb300.gemm import Gemm
from test_gpu_fp8_limits import limited

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = Gemm(torch.device("cuda", 0))
    yield g
    g.close()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K,tile", [(1, 4096, 4096, -1), (20, 4096, 4096, -1),
                                        (50, 4096, 4096, -1), (300, 700, 2048, -1),
                                        (2048, 2048, 2048, -1), (1024, 2048, 2048, 256),
                                        (4096, 4096, 1024, 256)])
def test_product_under_short_limits(h, M, N, K, tile, fmt):
    """Split over clusters, whole tiles of one CTA, and of CTA pairs, one and several each."""
    torch.manual_seed(M)
    a = h.fp4_quantize(torch.randn(M, K, device="cuda"), fmt)
    b = h.fp4_quantize(torch.randn(N, K, device="cuda"), fmt)
    h.set_option(B.GEMM_OPT_FORCE_TILE_N, tile)
    try:
        limited(h, lambda: [h.fp4_matmul(a, b)], [1, 300, 1000, 3000, 10000, 30000])
    finally:
        h.set_option(B.GEMM_OPT_FORCE_TILE_N, -1)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,split", [(1, -1), (1, 2), (20, 8), (50, 4)])
def test_swapped_product_under_short_limits(h, M, split, fmt):
    """One row kept on the tensor cores, and splits over 2, 4 and 8 CTAs."""
    torch.manual_seed(M)
    a = h.fp4_quantize(torch.randn(M, 4096, device="cuda"), fmt)
    b = h.fp4_quantize(torch.randn(1500, 4096, device="cuda"), fmt)
    h.set_option(B.GEMM_OPT_FORCE_SWAP_AB, 1)
    h.set_option(B.GEMM_OPT_CLUSTER_SPLIT, split)
    try:
        limited(h, lambda: [h.fp4_matmul(a, b)], [1, 300, 1000, 3000, 10000, 30000])
    finally:
        h.set_option(B.GEMM_OPT_FORCE_SWAP_AB, -1)
        h.set_option(B.GEMM_OPT_CLUSTER_SPLIT, -1)
