"""Torch-facing wrapper over the C-ABI: tensors -> pointers, sizes, layout and
the current CUDA stream.  PyTorch supplies device memory and streams only."""
from __future__ import annotations

import ctypes

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


_BOTH = ("row", "col")
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
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
        self._lib = B.load()
        self._run = self._lib.gemm_run  # argument types set once by the binding

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
    def _raw_stream(self, stream):
        """The stream's handle, without building a Stream object for the current
        one (2 us of a call's 10)."""
        return stream.cuda_stream if stream is not None else _current_raw(self.device.index)

    def fp8_quantize(self, x: torch.Tensor, blocks: str = "row", stream=None):
        """x (rows, cols; float16, bfloat16 or float32, unit stride along its
        rows) as an Fp8Matrix with "row", "col" or "tile" blocks, or, for
        "row+col", a pair of them from one pass over x."""
        code = _DT8.get(x.dtype)
        if code is None:
            raise TypeError("x must be float16, bfloat16 or float32, got %s" % x.dtype)
        if x.dim() != 2:
            raise ValueError("x must be 2-D")
        if x.get_device() != self.device.index:
            raise ValueError("tensor on %s, handle on %s" % (x.device, self.device))
        rows, cols = x.shape
        sr, sc = x.stride()
        if cols > 1 and sc != 1:
            raise ValueError("rows of x must be contiguous")
        if rows > 1 and sr < cols:
            raise ValueError("rows of x overlap")
        kinds = _BOTH if blocks == "row+col" else (blocks,)
        m = Fp8Matrix._carve(rows, cols, kinds, self.device)
        rc = self._lib.gemm_fp8_quantize(self.handle, rows, cols, x.data_ptr(),
                                         sr if sr > cols else cols, code, m[0].ref,
                                         m[1].ref if len(m) == 2 else None,
                                         self._raw_stream(stream))
        if rc != B.GEMM_OK:
            raise B.GemmError(rc, "gemm_fp8_quantize")
        return tuple(m) if len(m) == 2 else m[0]

    def fp8_run(self, A: Fp8Matrix, Bm: Fp8Matrix, C: torch.Tensor, bias=None, a_major=ROW,
                b_major=ROW, stream=None) -> None:
        """Enqueues C = A·B (+bias) of block-scaled matrices into C (M, N;
        float16, bfloat16 or float32, unit stride along its rows).  A is stored
        (M, K) row-major or (K, M) column-major, B (K, N) or (N, K); the blocks
        of each must run along K."""
        M, N, K = self._fp8_dims(A, Bm, a_major, b_major)
        if C.get_device() != self.device.index:
            raise ValueError("tensor on %s, handle on %s" % (C.device, self.device))
        code = _DT8.get(C.dtype)
        if code is None:
            raise TypeError("C must be float16, bfloat16 or float32, got %s" % C.dtype)
        if C.dim() != 2 or C.shape[0] != M or C.shape[1] != N:
            raise ValueError("C has shape %s, expected (%d, %d)" % (tuple(C.shape), M, N))
        sr, sc = C.stride()
        if (N > 1 and sc != 1) or (M > 1 and sr < N):
            raise ValueError("rows of C must be contiguous and not overlap")
        self._fp8_launch(M, N, K, A, Bm, bias, C, max(sr, N), a_major, b_major, code, stream)

    def _fp8_dims(self, A, Bm, a_major, b_major):
        """(M, N, K) of a product of two Fp8Matrix on this handle's device."""
        sa, sb = A.shape, Bm.shape
        if len(sa) != 2 or len(sb) != 2:
            raise ValueError("A and B must be 2-D")
        M, K = sa if a_major == ROW else (sa[1], sa[0])
        Kb, N = sb if b_major == ROW else (sb[1], sb[0])
        if K != Kb:
            raise ValueError("inner dimensions differ: %d vs %d" % (K, Kb))
        idx = self.device.index
        if A.device_index != idx or Bm.device_index != idx:
            raise ValueError("operands must be on the handle's device, %s" % self.device)
        return M, N, K

    def _fp8_launch(self, M, N, K, A, Bm, bias, C, ldc, a_major, b_major, code, stream):
        bias_ptr = None
        if bias is not None:
            if (bias.dtype != torch.float32 or tuple(bias.shape) != (N,)
                    or not bias.is_contiguous()):
                raise ValueError("bias must be contiguous float32 of shape (N,)")
            if bias.get_device() != self.device.index:
                raise ValueError("tensor on %s, handle on %s" % (bias.device, self.device))
            bias_ptr = bias.data_ptr()
        rc = self._lib.gemm_fp8_run(self.handle, M, N, K, A.ref, Bm.ref, bias_ptr, C.data_ptr(),
                                    ldc, a_major, b_major, code, self._raw_stream(stream))
        if rc != B.GEMM_OK:
            raise B.GemmError(rc, "gemm_fp8_run")

    def fp8_matmul(self, A: Fp8Matrix, Bm: Fp8Matrix, bias=None, a_major=ROW, b_major=ROW,
                   out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
        """A·B (+bias) as a new tensor (see fp8_run)."""
        M, N, K = self._fp8_dims(A, Bm, a_major, b_major)
        code = _DT8.get(out_dtype)
        if code is None:
            raise TypeError("out_dtype must be float16, bfloat16 or float32, got %s" % out_dtype)
        C = torch.empty((M, N), dtype=out_dtype, device=self.device)
        self._fp8_launch(M, N, K, A, Bm, bias, C, N, a_major, b_major, code, stream)
        return C

    def moe_fp8(self, x: torch.Tensor, router: torch.Tensor, gate: Fp8Matrix, up: Fp8Matrix,
                down: Fp8Matrix, top_k: int, renormalize: bool = True, stream=None):
        """A mixture-of-experts layer on a few tokens: x (tokens, hidden) and
        router (experts, hidden) float16 or bfloat16, gate and up Fp8Matrix
        (experts, inner, hidden), down (experts, hidden, inner).  Returns out
        (tokens, hidden), ids (tokens, top_k) int32 and gates (tokens, top_k)
        float32; the arithmetic is that of gemm_moe_fp8."""
        if x.dim() != 2 or router.dim() != 2 or router.shape[1] != x.shape[1]:
            raise ValueError("x must be (tokens, hidden), router (experts, hidden)")
        T, H = x.shape
        E = router.shape[0]
        if len(gate.shape) != 3 or len(up.shape) != 3 or len(down.shape) != 3:
            raise ValueError("gate, up and down must be (experts, rows, cols)")
        I = gate.shape[1]
        if (tuple(gate.shape) != (E, I, H) or tuple(up.shape) != (E, I, H)
                or tuple(down.shape) != (E, H, I)):
            raise ValueError("weights have shapes %s, %s and %s, expected gate and up (%d, inner, "
                             "%d), down (%d, %d, inner)" % (tuple(gate.shape), tuple(up.shape),
                                                            tuple(down.shape), E, H, E, H))
        if x.dtype != router.dtype or x.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("x and router: both float16 or both bfloat16")
        if not 1 <= top_k <= E:
            raise ValueError("top_k must be 1 ... %d, got %d" % (E, top_k))
        idx = self.device.index
        for d in (x.get_device(), router.get_device(), gate.device_index, up.device_index,
                  down.device_index):
            if d != idx:
                raise ValueError("operands must be on the handle's device, %s" % self.device)
        for t in (x, router):
            if (H > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < H):
                raise ValueError("rows of x and router must be contiguous")
        out = torch.empty((T, H), dtype=x.dtype, device=self.device)
        ids = torch.empty((T, top_k), dtype=torch.int32, device=self.device)
        gates = torch.empty((T, top_k), dtype=torch.float32, device=self.device)
        L = B.gemm_moe_fp8_t(T, H, I, E, top_k, 1 if renormalize else 0, _DT8[x.dtype], 0,
                             x.data_ptr(), max(x.stride(0), H), router.data_ptr(),
                             max(router.stride(0), H), gate.desc, up.desc, down.desc,
                             out.data_ptr(), H, ids.data_ptr(), gates.data_ptr())
        rc, n = B.gemm_moe_fp8_workspace(self.handle, L)
        if rc != B.GEMM_OK:
            raise B.GemmError(rc, "gemm_moe_fp8_workspace")
        s = self._raw_stream(stream)
        ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        if stream is not None:
            ws.record_stream(stream)
        rc = self._lib.gemm_moe_fp8(self.handle, ctypes.byref(L), ws.data_ptr(), n, s)
        if rc != B.GEMM_OK:
            raise B.GemmError(rc, "gemm_moe_fp8")
        return out, ids, gates
