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


# ------------------------------------------------------------ forms beside the plain ones --
def q_values(t, blocks):
    return R.values(*R.quantize(R.host(t), blocks), blocks)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_linear_with_bias_in_every_type(g, dtype):
    """y, dx, dW and the bias gradient against the formula on the quantised operands, dW
    in the weight's type."""
    torch.manual_seed(1)
    T, N, K = 75, 200, 330
    x = torch.randn(T, K).to(dtype).cuda().requires_grad_()
    w = (torch.randn(N, K) * K ** -0.5).to(dtype).cuda().requires_grad_()
    bias = torch.randn(N).cuda().requires_grad_()
    dy = torch.randn(T, N).to(dtype).cuda()
    y = fp8.linear(g, x, w, bias)
    y.backward(dy)
    g.status()
    b = R.host(bias)
    for got, A, Bm, add in ((y, q_values(x, "row"), q_values(w, "tile").T, b),
                            (x.grad, q_values(dy, "row"), q_values(w, "tile"), 0.0),
                            (w.grad, q_values(dy, "col").T, q_values(x, "col"), 0.0)):
        want = A @ Bm + add
        assert got.dtype == dtype
        bound = R.product_bound(A, Bm, want, dtype) + 2 * R.U32 * (np.abs(want) + np.abs(add))
        assert (np.abs(R.host(got) - want) <= bound).all()
    d = R.host(dy)
    assert (np.abs(R.host(bias.grad) - d.sum(0)) <= T * R.U32 * np.abs(d).sum(0)).all()


def test_linear_without_a_weight_gradient(g):
    torch.manual_seed(2)
    x = torch.randn(40, 256, device="cuda").bfloat16().requires_grad_()
    w = torch.randn(128, 256, device="cuda").bfloat16()
    both = w.clone().requires_grad_()
    fp8.linear(g, x, both).sum().backward()
    want, x.grad = x.grad, None
    fp8.linear(g, x, w).sum().backward()
    assert torch.equal(x.grad, want)


def expert_weights(rng, E, rows, cols):
    q = R.round_e4m3(np.clip(rng.standard_normal((E, rows, cols)) * 112, -448, 448))
    s = ((0.5 + rng.random((E, -(-rows // 128), -(-cols // 128)))) / (112 * cols ** 0.5)
         ).astype(np.float32)
    buf = torch.zeros(E, rows, -(-cols // 16) * 16, dtype=torch.uint8)
    buf[:, :, :cols] = torch.from_numpy(q).float().to(torch.float8_e4m3fn).view(torch.uint8)
    return (Fp8Matrix(buf.cuda()[:, :, :cols], torch.from_numpy(s).cuda(), "tile"),
            R.values(q, s, "tile"))


@pytest.mark.parametrize("T,H,I,E,k", [(5, 64, 48, 512, 16), (64, 64, 48, 512, 8),
                                       (33, 200, 130, 511, 3)])
def test_as_many_experts_as_there_may_be(g, T, H, I, E, k):
    rng = np.random.default_rng(E + T)
    (W1, w1), (W3, w3), (W2, w2) = (expert_weights(rng, E, *s) for s in ((I, H), (I, H), (H, I)))
    x = torch.from_numpy(rng.standard_normal((T, H))).to(BF16)
    router = torch.from_numpy(rng.standard_normal((E, H)) * H ** -0.5).to(BF16)
    out, ids, gates = g.moe_fp8(x.cuda(), router.cuda(), W1, W3, W2, k)
    g.status()
    ids = ids.cpu().numpy().astype(np.int64)
    R.check_choice(R.host(x), R.host(router), ids)
    want, slack, gv, e_g = R.moe(R.host(x), R.host(router), w1, w3, w2, ids, True)
    assert (np.abs(R.host(gates) - gv) <= e_g).all()
    bound = slack + R.OUT_U[BF16] * (np.abs(want) + slack) + R.OUT_TINY[BF16]
    assert (np.abs(R.host(out) - want) <= bound).all()


def test_a_token_s_choice_and_gates_do_not_depend_on_its_neighbours(g):
    """Its ids and gates bit for bit; its row of `out` within the bound (the sums may be
    cut elsewhere)."""
    rng = np.random.default_rng(14)
    T, H, I, E, k = 19, 520, 300, 24, 4
    (W1, w1), (W3, w3), (W2, w2) = (expert_weights(rng, E, *s) for s in ((I, H), (I, H), (H, I)))
    x = torch.from_numpy(rng.standard_normal((T, H))).to(BF16).cuda()
    router = torch.from_numpy(rng.standard_normal((E, H)) * H ** -0.5).to(BF16).cuda()
    out, ids, gates = g.moe_fp8(x, router, W1, W3, W2, k)
    want, slack, _, _ = R.moe(R.host(x), R.host(router), w1, w3, w2,
                              ids.cpu().numpy().astype(np.int64), True)
    bound = slack + R.OUT_U[BF16] * (np.abs(want) + slack) + R.OUT_TINY[BF16]
    for first, last in ((0, 1), (7, 8), (18, 19), (3, 12)):
        o, i, p = g.moe_fp8(x[first:last], router, W1, W3, W2, k)
        assert torch.equal(i, ids[first:last]) and torch.equal(p, gates[first:last])
        assert (np.abs(R.host(o) - want[first:last]) <= bound[first:last]).all()
    g.status()


def test_two_handles_in_two_threads():
    """A handle and a stream for each of two threads, products and expert layers at
    the same time: the same bits as one after the other."""
    import threading

    rng = np.random.default_rng(8)
    E, H, I, k = 8, 512, 256, 2
    ws = [expert_weights(rng, E, *s)[0] for s in ((I, H), (I, H), (H, I))]
    handles = [Gemm(torch.device("cuda", 0)) for _ in range(2)]
    router = torch.randn(E, H, device="cuda").half()
    data = [(torch.randn(100, H, device="cuda").half(), torch.randn(300, H, device="cuda").half())
            for _ in range(2)]

    def work(h, x, w):
        a, b = h.fp8_quantize(x, "row"), h.fp8_quantize(w, "tile")
        return (h.fp8_matmul(a, b, b_major=COL),) + h.moe_fp8(x[:9], router, *ws, k)

    want = [work(h, *d) for h, d in zip(handles, data)]
    torch.cuda.synchronize()
    failed = []

    def thread(n):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(30):
                    got = work(handles[n], *data[n])
                    s.synchronize()
                    assert all(torch.equal(a, b) for a, b in zip(got, want[n]))
        except BaseException as e:  # shown by the test's own thread
            failed.append(e)

    threads = [threading.Thread(target=thread, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for h in handles:
        h.status()
        h.close()
    assert not failed, failed


def test_calls_in_a_row_on_a_busy_stream(g):
    """Quantise, product and quantise again behind a delay, without a graph and without
    waiting between: each reads what the one before wrote."""
    torch.manual_seed(6)
    x = torch.randn(64, 512, device="cuda").bfloat16()
    ws = [g.fp8_quantize(torch.randn(512, 512, device="cuda") * 512 ** -0.5, "tile")
          for _ in range(6)]

    def chain(wait):
        y = x
        for w in ws:
            y = g.fp8_matmul(g.fp8_quantize(y, "row"), w, b_major=COL)
            if wait:
                torch.cuda.synchronize()
        return y

    want = chain(True)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(5):
            torch.cuda._sleep(5_000_000)
            got = [chain(False) for _ in range(3)]
            s.synchronize()
            assert all(torch.equal(y, want) for y in got)
    g.status()


def test_a_given_stream_in_a_capture(g):
    """The calls with stream= inside a graph's capture on that stream, inputs from another."""
    torch.manual_seed(9)
    x, w = torch.randn(50, 384, device="cuda").half(), torch.randn(200, 384, device="cuda").half()
    wq = g.fp8_quantize(w, "tile")
    want = g.fp8_matmul(g.fp8_quantize(x, "row"), wq, b_major=COL)
    C = torch.empty_like(want)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        xq = g.fp8_quantize(x, "row", stream=s)
        y = g.fp8_matmul(xq, wq, b_major=COL, stream=s)
        g.fp8_run(xq, wq, C, b_major=COL, stream=s)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(C, want)
    g.status()
