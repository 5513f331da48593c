"""The 8-bit operators under wait limits short enough to run out anywhere in a
launch: it ends, gemm_status reports it or the result is right, and the next call
is right."""
import pytest
import torch

from dense_gemm_tmem_gb300 import binding as B
from dense_gemm_tmem_gb300.fp8 import Fp8Matrix
from dense_gemm_tmem_gb300.gemm import Gemm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = Gemm(torch.device("cuda", 0))
    yield g
    g.close()


def limited(h, call, limits, times=8):
    """`call`'s tensors, bit for bit, whatever happened to the limited calls before."""
    want = call()
    h.status()
    stream = torch.cuda.current_stream().cuda_stream
    for ns in limits:
        for _ in range(times):
            h.set_option(B.GEMM_OPT_WAIT_LIMIT_NS, ns)
            try:
                got = call()
                rc = B.gemm_status(h.handle, stream)
            finally:
                h.set_option(B.GEMM_OPT_WAIT_LIMIT_NS, -1)
            assert rc in (B.GEMM_OK, B.GEMM_ERR_DEVICE_TIMEOUT)
            if rc == B.GEMM_OK:
                assert all(torch.equal(a, b) for a, b in zip(got, want))
            assert all(torch.equal(a, b) for a, b in zip(call(), want))
            h.status()


def experts(count, rows, cols):
    torch.manual_seed(rows)
    data = torch.randint(0, 127, (count, rows, cols), dtype=torch.uint8, device="cuda")
    scale = torch.rand(count, -(-rows // 128), -(-cols // 128), device="cuda") * 1e-3
    return Fp8Matrix(data, scale, "tile")


@pytest.mark.parametrize("tokens,hidden,inner,count,top_k",
                         [(1, 512, 256, 8, 2), (16, 1024, 512, 16, 4), (64, 2048, 1024, 64, 4)])
def test_expert_layer_under_short_limits(h, tokens, hidden, inner, count, top_k):
    w = (experts(count, inner, hidden), experts(count, inner, hidden),
         experts(count, hidden, inner))
    torch.manual_seed(1)
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    router = torch.randn(count, hidden, device="cuda").bfloat16()
    limited(h, lambda: h.moe_fp8(x, router, *w, top_k), [1, 300, 1000, 3000, 10000, 30000])


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (300, 700, 2048), (2048, 2048, 2048)])
def test_product_under_short_limits(h, M, N, K):
    """Split over clusters, whole tiles of one wave, and several tiles a CTA."""
    torch.manual_seed(M)
    a = h.fp8_quantize(torch.randn(M, K, device="cuda").half(), "row")
    b = h.fp8_quantize(torch.randn(N, K, device="cuda").half(), "tile")
    limited(h, lambda: [h.fp8_matmul(a, b, b_major=B.GEMM_COL_MAJOR)], [1, 300, 1000, 3000, 10000])
