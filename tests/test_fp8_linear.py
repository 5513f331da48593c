"""The differentiable linear layer's bookkeeping, on the host: what it keeps for the
backward pass and which of its quantisations and products it asks for, seen by a
stand-in for the library handle that computes them in plain torch."""
import gc
import itertools
import weakref

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import fp8_reference as R
from dense_gemm_tmem_gb300 import fp8
from dense_gemm_tmem_gb300.fp8 import Fp8Matrix
from dense_gemm_tmem_gb300.gemm import COL, ROW

BF16, F32 = torch.bfloat16, torch.float32


class Plain:
    """fp8_quantize and fp8_matmul of a Gemm, noting each call."""

    def __init__(self):
        self.calls, self.made = [], []

    def fp8_quantize(self, x, blocks="row", stream=None):
        self.calls.append(blocks)
        out = []
        for kind in blocks.split("+"):
            q, s = R.quantize(R.host(x), kind)
            out.append(Fp8Matrix(torch.from_numpy(q).float().to(torch.float8_e4m3fn),
                                 torch.from_numpy(s), kind))
            self.made.append((kind, weakref.ref(out[-1].data)))
        return tuple(out) if len(out) == 2 else out[0]

    def fp8_matmul(self, A, Bm, bias=None, a_major=ROW, b_major=ROW, out_dtype=BF16, stream=None):
        self.calls.append((tuple(A.shape), tuple(Bm.shape), out_dtype))
        a, b = A.dequantize().double(), Bm.dequantize().double()
        c = (a if a_major == ROW else a.t()) @ (b if b_major == ROW else b.t())
        return (c if bias is None else c + bias.double()).to(out_dtype)

    def products(self):
        return [c for c in self.calls if isinstance(c, tuple)]


T, N, K = 5, 6, 7


def leaves(need_x=True, need_w=True, need_b=True, dtype=F32):
    torch.manual_seed(0)
    return (torch.randn(T, K).to(dtype).requires_grad_(need_x),
            torch.randn(N, K).to(dtype).requires_grad_(need_w),
            torch.randn(N).requires_grad_(need_b))


def alive(g, kind):
    gc.collect()
    return [i for i, (k, r) in enumerate(g.made) if k == kind and r() is not None]


def test_nothing_is_kept_after_the_backward_pass():
    g = Plain()
    x, w, bias = leaves()
    y = fp8.linear(g, x, w, bias)
    assert alive(g, "col") and alive(g, "tile")
    assert not alive(g, "row")  # the forward product's own copy
    y.sum().backward()
    assert not alive(g, "col") and not alive(g, "tile")  # y is alive still
    with pytest.raises(RuntimeError):
        y.sum().backward()
    y2 = fp8.linear(g, x, w, bias)
    y2.sum().backward(retain_graph=True)
    x.grad = None
    y2.sum().backward(retain_graph=True)
    first, x.grad = x.grad, None
    y2.sum().backward()
    assert torch.equal(x.grad, first)


@pytest.mark.parametrize("need", list(itertools.product([False, True], repeat=3)))
def test_only_what_is_needed_is_computed_and_kept(need):
    """Each combination of x, w and bias that require a gradient: the same values as
    with all of them, and no quantisation, product or kept copy beside."""
    need_x, need_w, need_b = need
    whole = leaves()
    fp8.linear(Plain(), *whole).square().sum().backward()
    g = Plain()
    some = leaves(*need)
    y = fp8.linear(g, *some)
    assert g.calls == ["row+col" if need_w else "row", "tile", ((T, K), (N, K), F32)]
    assert bool(alive(g, "col")) == need_w and bool(alive(g, "tile")) == need_x
    assert not alive(g, "row")
    if not any(need):
        assert not y.requires_grad
        return
    g.calls.clear()
    y.square().sum().backward()
    want = {(True, True): ["row+col"], (True, False): ["row"], (False, True): ["col"],
            (False, False): []}[need_x, need_w]
    assert [c for c in g.calls if isinstance(c, str)] == want
    assert len(g.products()) == need_x + need_w
    for a, b, n in zip(some, whole, need):
        assert (a.grad is not None) == n
        if n:
            assert torch.equal(a.grad, b.grad)


def test_without_a_graph_nothing_is_kept():
    g = Plain()
    with torch.no_grad():
        y = fp8.linear(g, *leaves())
    assert not y.requires_grad and g.calls[0] == "row"
    assert not alive(g, "tile")


def test_backward_refuses_what_forward_was_told_to_drop():
    g = Plain()
    x, w, _ = (t.detach() for t in leaves())
    y, saved = fp8.linear_forward(g, x, w, need_dw=False)
    assert saved[0] is None
    dx, dw = fp8.linear_backward(g, y, saved, need_dw=False)
    assert dw is None and dx.shape == x.shape
    with pytest.raises(ValueError):
        fp8.linear_backward(g, y, saved)


@pytest.mark.parametrize("dtype", [torch.float16, BF16, F32])
def test_the_weight_gradient_is_asked_for_in_the_weight_s_type(dtype):
    """One rounding of the fp32 sums, not a product in fp32 and a pass that casts it."""
    g = Plain()
    x, w, bias = leaves(dtype=dtype)
    y = fp8.linear(g, x, w, bias)
    g.calls.clear()
    y.sum().backward()
    assert [c[2] for c in g.products()] == [dtype, dtype]
    assert w.grad.dtype == dtype and bias.grad.dtype == F32


@pytest.mark.parametrize("dtype", [torch.float16, BF16])
def test_the_bias_gradient_makes_no_copy_of_dy(dtype):
    x, w, bias = leaves(False, False, True, dtype)
    y = fp8.linear(Plain(), x, w, bias)
    dy, seen = torch.randn(T, N).to(dtype), []
    with Seen(seen):
        y.backward(dy)
    assert not any(shape == (T, N) and t == F32 for _, shape, t in seen)
    assert torch.equal(bias.grad, dy.float().sum(0))


class Seen(TorchDispatchMode):
    """Notes what runs and what it makes."""

    def __init__(self, out):
        super().__init__()
        self.out = out

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        r = func(*args, **(kwargs or {}))
        if isinstance(r, torch.Tensor):
            self.out.append((func._schema.name, tuple(r.shape), r.dtype))
        return r
