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


def test_inputs_may_be_dropped_while_a_busy_stream_reads_them(g):
    """A call on another stream is still queued when it returns: what it reads, made
    on the current stream and dropped, must not be handed out again before."""
    torch.manual_seed(3)
    T, N, K = 256, 384, 512
    x, w, dy = (torch.randn(*s, device="cuda").bfloat16() for s in ((T, K), (N, K), (T, N)))
    want_q = g.fp8_quantize(x, "row")
    wq = g.fp8_quantize(w, "tile")
    want_y = g.fp8_matmul(want_q, wq, b_major=COL)
    want = fp8.linear_backward(g, dy, fp8.linear_forward(g, x, w)[1])
    s = torch.cuda.Stream()

    def junk():  # what the current stream's next tensors write
        return [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")
                for n in (2 * T * K, T * K + 4 * T * 4, T * K + 4 * 2 * K, N * K + 4 * 3 * 4,
                          2 * T * N, 2 * T * N) for _ in range(3)]

    def busy():
        torch.cuda.synchronize()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)

    for _ in range(3):
        xs = x.clone()
        busy()
        q = g.fp8_quantize(xs, "row", stream=s)
        del xs
        keep = junk()
        torch.cuda.synchronize()
        assert torch.equal(q.data.view(torch.uint8), want_q.data.view(torch.uint8))
        del keep

        a, b = g.fp8_quantize(x, "row"), g.fp8_quantize(w, "tile")
        busy()
        y = g.fp8_matmul(a, b, b_major=COL, stream=s)
        del a, b
        keep = junk()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y)
        del keep

        a, b = g.fp8_quantize(x, "row"), g.fp8_quantize(w, "tile")
        C = torch.empty(T, N, dtype=BF16, device="cuda")
        busy()
        g.fp8_run(a, b, C, b_major=COL, stream=s)
        del a, b
        keep = junk()
        torch.cuda.synchronize()
        assert torch.equal(C, want_y)
        del keep

        saved, d = fp8.linear_forward(g, x, w)[1], dy.clone()
        busy()
        got = fp8.linear_backward(g, d, saved, stream=s)
        del saved, d
        keep = junk()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        del keep
    g.status()


def test_expert_layer_s_inputs_may_be_dropped(g):
    rng = np.random.default_rng(5)
    T, H, I, E, k = 6, 256, 128, 8, 2

    def experts(rows, cols):
        q = R.round_e4m3(np.clip(rng.standard_normal((E, rows, cols)) * 112, -448, 448))
        return (torch.from_numpy(q).float().to(torch.float8_e4m3fn).cuda(),
                torch.full((E, rows // 128, cols // 128), 1e-3, device="cuda"))

    parts = [experts(*s) for s in ((I, H), (I, H), (H, I))]
    x = torch.randn(T, H, device="cuda").half()
    router = torch.randn(E, H, device="cuda").half()
    want = g.moe_fp8(x, router, *(Fp8Matrix(*p, "tile") for p in parts), k)
    s = torch.cuda.Stream()
    for _ in range(3):
        own = [x.clone(), router.clone()]
        ws = [Fp8Matrix(d.clone(), c.clone(), "tile") for d, c in parts]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        got = g.moe_fp8(*own, *ws, k, stream=s)
        del own, ws
        keep = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")
                for n in (2 * T * H, 2 * E * H, E * I * H, 4 * E * 2) for _ in range(4)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del keep
    g.status()
