"""Torch-facing wrapper over the C-ABI: tensors -> pointers, sizes, layout and
the current CUDA stream.  PyTorch supplies device memory and streams only."""
from __future__ import annotations

import torch

from . import binding as B
from .fp8 import Fp8Matrix

_DT = {torch.float16: B.GEMM_F16, torch.float32: B.GEMM_F32}
_DT8 = {**_DT, torch.bfloat16: B.GEMM_BF16}  # the 8-bit operators' other types
ROW, COL = B.GEMM_ROW_MAJOR, B.GEMM_COL_MAJOR


def problem_dims(A: torch.Tensor, Bm: torch.Tensor, a_major: int, b_major: int):
    """(M, N, K) from storage tensors: A is (M, K) row-major or (K, M)
    column-major; B is (K, N) row-major or (N, K) column-major."""
    if A.dim() != 2 or Bm.dim() != 2:
        raise ValueError("A and B must be 2-D")
    M, K = (A.shape[0], A.shape[1]) if a_major == ROW else (A.shape[1], A.shape[0])
    Kb, N = (Bm.shape[0], Bm.shape[1]) if b_major == ROW else (Bm.shape[1], Bm.shape[0])
    if K != Kb:
        raise ValueError("inner dimensions differ: %d vs %d" % (K, Kb))
    return int(M), int(N), int(K)


_KINDS = {"row": (B.GEMM_FP8_ROW, -1), "col": (B.GEMM_FP8_COL, -1),
          "tile": (B.GEMM_FP8_TILE, -1), "row+col": (B.GEMM_FP8_ROW, B.GEMM_FP8_COL)}
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _in_use(stream, *tensors):
    """The allocator keeps the tensors' memory until the stream has passed this point,
    though they are another stream's and may be dropped meanwhile."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


_LAYOUTS = {}  # (a_major, b_major, in, out) -> gemm_layout_t, built once


def _layout(a_major, b_major, in_code, out_code):
    key = (a_major, b_major, in_code, out_code)
    lay = _LAYOUTS.get(key)
    if lay is None:
        lay = _LAYOUTS[key] = B.layout(a_major, b_major, in_code, out_code)
    return lay


class Gemm:
    """One library handle on one CUDA device."""

    def __init__(self, device=0):
        dev = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
        if dev.index is None:
            dev = torch.device("cuda", 0)
        self.device = dev
        self.handle = B.gemm_create(dev.index)
        self._native = None  # the extension, once an 8-bit call has been made
        self._run = B.load().gemm_run  # argument types set once by the binding

    def close(self):
        if getattr(self, "handle", None):
            torch.cuda.synchronize(self.device)
            B.gemm_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            if getattr(self, "handle", None):
                B.gemm_destroy(self.handle)
                self.handle = None
        except Exception:
            pass

    def _stream(self, stream):
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        return s.cuda_stream

    def layout(self, A, Bm, C, a_major, b_major):
        return _layout(a_major, b_major, _DT[A.dtype], _DT[C.dtype])

    def run(self, A, Bm, C, bias=None, a_major=ROW, b_major=ROW, stream=None) -> None:
        """Enqueues C = A·B (+bias) into the preallocated row-major C."""
        M, N, K = problem_dims(A, Bm, a_major, b_major)
        idx = self.device.index
        for t in (A, Bm, C) + ((bias,) if bias is not None else ()):
            if t.get_device() != idx:
                raise ValueError("tensor on %s, handle on %s" % (t.device, self.device))
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")
        in_code, out_code = _DT.get(A.dtype), _DT.get(C.dtype)
        if A.dtype != Bm.dtype or in_code is None or out_code is None:
            raise TypeError("A, B: both float16 or both float32; C: float16 or float32")
        if C.dim() != 2 or C.shape[0] != M or C.shape[1] != N:
            raise ValueError("C has shape %s, expected (%d, %d)" % (tuple(C.shape), M, N))
        if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (N,)):
            raise ValueError("bias must be float32 of shape (N,)")
        rc = self._run(self.handle, M, N, K, A.data_ptr(), Bm.data_ptr(),
                       bias.data_ptr() if bias is not None else None, C.data_ptr(),
                       _layout(a_major, b_major, in_code, out_code), self._stream(stream))
        if rc != B.GEMM_OK:
            raise B.GemmError(rc, "gemm_run")

    def run_host(self, A, Bm, C, bias=None, a_major=ROW, b_major=ROW, stream=None) -> None:
        """Enqueues C = A·B (+bias) on host (CPU) tensors through gemm_run_host:
        copies in, the GEMM and the copy out all on the stream.  Pinned tensors
        (`.pin_memory()`) make the copies asynchronous; C is ready once the
        stream has reached this point (e.g. after `status()`), and every
        tensor passed must stay alive until then."""
        M, N, K = problem_dims(A, Bm, a_major, b_major)
        for t in (A, Bm, C) + ((bias,) if bias is not None else ()):
            if t.device.type != "cpu":
                raise ValueError("run_host takes host tensors; got one on %s" % t.device)
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")
        in_code, out_code = _DT.get(A.dtype), _DT.get(C.dtype)
        if A.dtype != Bm.dtype or in_code is None or out_code is None:
            raise TypeError("A, B: both float16 or both float32; C: float16 or float32")
        if C.dim() != 2 or C.shape[0] != M or C.shape[1] != N:
            raise ValueError("C has shape %s, expected (%d, %d)" % (tuple(C.shape), M, N))
        if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (N,)):
            raise ValueError("bias must be float32 of shape (N,)")
        rc = B.gemm_run_host(self.handle, M, N, K, A.data_ptr(), Bm.data_ptr(),
                             bias.data_ptr() if bias is not None else None, C.data_ptr(),
                             _layout(a_major, b_major, in_code, out_code), self._stream(stream))
        if rc != B.GEMM_OK:
            raise B.GemmError(rc, "gemm_run_host")

    def __call__(self, A, Bm, bias=None, a_major=ROW, b_major=ROW, out_dtype=torch.float32,
                 stream=None) -> torch.Tensor:
        M, N, _ = problem_dims(A, Bm, a_major, b_major)
        C = torch.empty((M, N), dtype=out_dtype, device=self.device)
        self.run(A, Bm, C, bias, a_major, b_major, stream)
        return C

    def status(self, stream=None) -> None:
        """Synchronises the stream and raises if a device-side wait expired."""
        rc = B.gemm_status(self.handle, self._stream(stream))
        if rc != B.GEMM_OK:
            raise B.GemmError(rc, "gemm_status (detail %d)" % B.gemm_status_detail(self.handle))

    def set_option(self, option: int, value: int) -> None:
        rc = B.gemm_set_option(self.handle, option, value)
        if rc != B.GEMM_OK:
            raise B.GemmError(rc, "gemm_set_option")

    def plan(self, M, N, K, a_major=ROW, b_major=ROW, in_dtype=B.GEMM_F16,
             out_dtype=B.GEMM_F32) -> dict:
        rc, p = B.gemm_query_plan(self.handle, M, N, K,
                                  B.layout(a_major, b_major, in_dtype, out_dtype))
        if rc != B.GEMM_OK:
            raise B.GemmError(rc, "gemm_query_plan")
        return p.as_dict()

    # ---- block-scaled 8-bit operators (include/gemm_fp8.h)
    def _extension(self):
        """The extension, which only these calls need: loaded at the first of them."""
        self._native = B.native()
        return self._native

    def _raw_stream(self, stream):
        """The stream's handle, without building a Stream object for the current
        one (2 us of a call's 10)."""
        return stream.cuda_stream if stream is not None else _current_raw(self.device.index)

    def fp8_quantize(self, x: torch.Tensor, blocks: str = "row", stream=None):
        """x (rows, cols; float16, bfloat16 or float32, unit stride along its
        rows) as an Fp8Matrix with "row", "col" or "tile" blocks, or, for
        "row+col", a pair of them from one pass over x.  With a stream, here and
        in fp8_run, fp8_matmul and moe_fp8, the tensors that the call makes are
        allocated on it, and those that it is given may be dropped at once;
        order it after what wrote the inputs.  None of them is differentiable:
        their results carry no gradient, whatever the inputs require
        (fp8.linear differentiates)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                r = self.fp8_quantize(x, blocks)
            _in_use(stream, x)
            return r
        kinds = _KINDS.get(blocks)
        if kinds is None:
            raise ValueError("blocks must be 'row', 'col', 'tile' or 'row+col', got %r"
                             % (blocks,))
        native = self._native or self._extension()
        r = native.quantize(self.handle, self.device.index, x, kinds[0], kinds[1],
                            _current_raw(self.device.index))
        if r.__class__ is int:
            raise B.GemmError(r, "gemm_fp8_quantize")
        if len(r) == 4:
            return Fp8Matrix._wrap(r[0], r[1], "row"), Fp8Matrix._wrap(r[2], r[3], "col")
        return Fp8Matrix._wrap(r[0], r[1], blocks)

    def fp8_run(self, A: Fp8Matrix, Bm: Fp8Matrix, C: torch.Tensor, bias=None, a_major=ROW,
                b_major=ROW, stream=None) -> None:
        """Enqueues C = A·B (+bias) of block-scaled matrices into C (M, N;
        float16, bfloat16 or float32, unit stride along its rows).  A is stored
        (M, K) row-major or (K, M) column-major, B (K, N) or (N, K); the blocks
        of each must run along K."""
        native = self._native or self._extension()
        rc = native.run(self.handle, self.device.index, A.data, A.scale, A.kind, Bm.data,
                        Bm.scale, Bm.kind, bias, a_major, b_major, C, self._raw_stream(stream))
        if rc != B.GEMM_OK:
            raise B.GemmError(rc, "gemm_fp8_run")
        if stream is not None:
            _in_use(stream, A.data, A.scale, Bm.data, Bm.scale, bias, C)

    def fp8_matmul(self, A: Fp8Matrix, Bm: Fp8Matrix, bias=None, a_major=ROW, b_major=ROW,
                   out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
        """A·B (+bias) as a new tensor (see fp8_run), which carries no gradient."""
        if stream is not None:
            with torch.cuda.stream(stream):
                C = self.fp8_matmul(A, Bm, bias, a_major, b_major, out_dtype)
            _in_use(stream, A.data, A.scale, Bm.data, Bm.scale, bias)
            return C
        code = _DT8.get(out_dtype)
        if code is None:
            raise TypeError("out_dtype must be float16, bfloat16 or float32, got %s" % out_dtype)
        native = self._native or self._extension()
        C = native.matmul(self.handle, self.device.index, A.data, A.scale, A.kind, Bm.data,
                          Bm.scale, Bm.kind, bias, a_major, b_major, code,
                          _current_raw(self.device.index))
        if C.__class__ is int:
            raise B.GemmError(C, "gemm_fp8_run")
        return C

    def moe_fp8(self, x: torch.Tensor, router: torch.Tensor, gate: Fp8Matrix, up: Fp8Matrix,
                down: Fp8Matrix, top_k: int, renormalize: bool = True, stream=None):
        """A mixture-of-experts layer on a few tokens: x (tokens, hidden) and
        router (experts, hidden) float16 or bfloat16, gate and up Fp8Matrix
        (experts, inner, hidden), down (experts, hidden, inner).  Returns out
        (tokens, hidden), ids (tokens, top_k) int32 and gates (tokens, top_k)
        float32, without gradients; the arithmetic is that of gemm_moe_fp8."""
        if stream is not None:
            with torch.cuda.stream(stream):
                r = self.moe_fp8(x, router, gate, up, down, top_k, renormalize)
            _in_use(stream, x, router, *(t for w in (gate, up, down) for t in (w.data, w.scale)))
            return r
        native = self._native or self._extension()
        r = native.moe(self.handle, self.device.index, x, router, gate.data, gate.scale, up.data,
                       up.scale, down.data, down.scale, top_k, 1 if renormalize else 0,
                       _current_raw(self.device.index))
        if r.__class__ is int:
            raise B.GemmError(r, "gemm_moe_fp8")
        return r
