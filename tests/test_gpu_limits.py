"""The fp16 tensor-core kernels under wait limits short enough to run out anywhere in
a launch: it ends, gemm_status reports it or the result is right, and the next call
is right."""
import pytest
import torch

from dense_gemm_tmem_gb300 import binding as B
from dense_gemm_tmem_gb300.gemm import COL, ROW, Gemm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = Gemm(torch.device("cuda", 0))
    yield g
    g.close()


# one tile of 64 and of 128 rows, split over a cluster, a wave of single CTAs, CTA pairs
@pytest.mark.parametrize("M,N,K", [(64, 64, 512), (128, 128, 1024), (16, 4096, 4096),
                                   (1000, 1100, 2048), (2048, 2048, 2048)])
def test_product_under_short_limits(h, M, N, K):
    torch.manual_seed(M)
    a = torch.randn(M, K, device="cuda").half()
    b = torch.randn(N, K, device="cuda").half()
    want, got = (torch.empty(M, N, device="cuda", dtype=torch.half) for _ in range(2))
    h.run(a, b, want, None, ROW, COL)
    h.status()
    stream = torch.cuda.current_stream().cuda_stream
    for ns in (1, 300, 1000, 3000, 10000):
        for _ in range(8):
            h.set_option(B.GEMM_OPT_WAIT_LIMIT_NS, ns)
            try:
                h.run(a, b, got, None, ROW, COL)
                rc = B.gemm_status(h.handle, stream)
            finally:
                h.set_option(B.GEMM_OPT_WAIT_LIMIT_NS, -1)
            assert rc in (B.GEMM_OK, B.GEMM_ERR_DEVICE_TIMEOUT)
            if rc == B.GEMM_OK:
                assert torch.equal(got, want)
            h.run(a, b, got, None, ROW, COL)
            h.status()
            assert torch.equal(got, want)
