"""Block-scaled 8-bit matrices and the layers built on them.

``Fp8Matrix`` holds what `Gemm.fp8_quantize` writes and `Gemm.fp8_matmul` and
`Gemm.moe_fp8` read: e4m3 values with one fp32 scale for each block of 128
(``"row"`` 1 x 128, ``"col"`` 128 x 1, ``"tile"`` 128 x 128).  ``linear_forward``
and ``linear_backward`` are the three products of a linear layer on them, and
``linear`` the same as a differentiable function.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as B

BLOCK = 128
BLOCKS = {"row": B.GEMM_FP8_ROW, "col": B.GEMM_FP8_COL, "tile": B.GEMM_FP8_TILE}
_BYTES = (torch.float8_e4m3fn, torch.uint8)
_byref, _new = ctypes.byref, object.__new__


def scale_shape(rows: int, cols: int, blocks: str):
    """Scales of a rows x cols matrix: one per block, the last ones ragged."""
    if blocks == "row":
        return rows, (cols + 127) >> 7
    if blocks == "tile":
        return (rows + 127) >> 7, (cols + 127) >> 7
    if blocks == "col":
        return (rows + 127) >> 7, cols
    raise ValueError("blocks must be 'row', 'col' or 'tile', got %r" % (blocks,))


class Fp8Matrix:
    """An e4m3 matrix (rows, cols), or one per expert (experts, rows, cols; tile
    blocks), with its scales.  ``data`` has unit stride along its rows; rows may
    be padded (``fp8_quantize`` pads them to 16 bytes, which the tensor cores
    need).  ``scale`` may have any strides.  The tensors are referenced, not
    copied; replacing them in place is seen by later calls."""

    __slots__ = ("blocks", "desc", "ref", "device_index", "shape", "_data", "_scale", "_buf",
                 "_layout")

    def __init__(self, data: torch.Tensor, scale: torch.Tensor, blocks: str):
        if data.dtype not in _BYTES:
            raise TypeError("data must be float8_e4m3fn (or its bytes as uint8), got %s"
                            % data.dtype)
        if scale.dtype != torch.float32:
            raise TypeError("scale must be float32, got %s" % scale.dtype)
        shape, st = data.shape, data.stride()
        if len(shape) not in (2, 3):
            raise ValueError("data must be 2-D, or 3-D with one matrix per expert")
        rows, cols = shape[-2:]
        if cols > 1 and st[-1] != 1:
            raise ValueError("rows of data must be contiguous")
        ld = st[-2] if rows > 1 else max(st[-2], cols)
        if ld < cols:
            raise ValueError("rows of data overlap")
        want = scale_shape(rows, cols, blocks)
        if len(shape) == 3:
            if blocks != "tile":
                raise ValueError("expert weights have tile blocks")
            want = (shape[0],) + want
        if tuple(scale.shape) != want:
            raise ValueError("scale has shape %s, expected %s" % (tuple(scale.shape), want))
        dev = data.get_device()
        if scale.get_device() != dev:
            raise ValueError("data on %s, scale on %s" % (data.device, scale.device))
        self._data, self._scale, self.blocks, self.device_index = data, scale, blocks, dev
        self.shape = shape
        ss = scale.stride()
        if len(shape) == 3:
            self.desc = B.gemm_fp8_experts_t(data.data_ptr(), ld, st[0], scale.data_ptr(), *ss)
            self.ref = None
        else:
            self.desc = B.gemm_fp8_matrix_t(data.data_ptr(), ld, scale.data_ptr(), ss[0], ss[1],
                                            BLOCKS[blocks], 0)
            self.ref = _byref(self.desc)

    @staticmethod
    def empty(rows: int, cols: int, blocks: str, device) -> "Fp8Matrix":
        """Unwritten storage in one allocation: rows padded to 16 bytes; the
        scales of 1 x 128 blocks with those of one k-block next to each other
        (the order the product's threads read them in), others row-major."""
        return Fp8Matrix._carve(rows, cols, (blocks,), device)[0]

    @staticmethod
    def _carve(rows, cols, kinds, device):
        """One unwritten matrix per block shape, all in one allocation."""
        ld = (cols + 15) & -16
        values = (rows * ld + 255) & -256
        parts, total = [], 0
        for blocks in kinds:
            shape = scale_shape(rows, cols, blocks)
            parts.append((blocks, shape, total))
            total += values + ((4 * shape[0] * shape[1] + 255) & -256)
        buf = torch.empty(total, dtype=torch.uint8, device=device)
        ptr, index = buf.data_ptr(), buf.get_device()
        out = []
        for blocks, shape, at in parts:
            m = _new(Fp8Matrix)
            m._data = m._scale = None  # made when first asked for
            strides = (1, shape[0]) if blocks == "row" else (shape[1], 1)
            m._buf, m._layout = buf, (ld, shape, strides, at, at + values)
            m.blocks, m.device_index, m.shape = blocks, index, (rows, cols)
            m.desc = B.gemm_fp8_matrix_t(ptr + at, ld, ptr + at + values, strides[0], strides[1],
                                         BLOCKS[blocks], 0)
            m.ref = _byref(m.desc)
            out.append(m)
        return out

    @property
    def data(self) -> torch.Tensor:
        """The e4m3 values (uint8 if the matrix was made from bytes)."""
        if self._data is None:
            ld, _, _, at, _ = self._layout
            self._data = self._buf.view(torch.float8_e4m3fn).as_strided(self.shape, (ld, 1), at)
        return self._data

    @property
    def scale(self) -> torch.Tensor:
        """The fp32 scales, one per block."""
        if self._scale is None:
            _, shape, strides, _, at = self._layout
            self._scale = self._buf.view(torch.float32).as_strided(shape, strides, at // 4)
        return self._scale

    def dequantize(self) -> torch.Tensor:
        """fp32 values, in plain torch (for checks and small matrices)."""
        r, c = self.data.shape[-2:]
        s = self.scale
        if self.blocks != "row":
            s = s.repeat_interleave(BLOCK, -2)[..., :r, :]
        if self.blocks != "col":
            s = s.repeat_interleave(BLOCK, -1)[..., :c]
        return self.data.view(torch.float8_e4m3fn).float() * s


def linear_forward(g, x: torch.Tensor, w, bias: torch.Tensor | None = None, stream=None):
    """y = x·Wᵀ (+bias) in 8 bits, and what linear_backward needs: x (tokens,
    inputs) is quantised along both axes in one pass, w is (outputs, inputs) or
    an Fp8Matrix of it with tile blocks.  y has x's type."""
    x_row, x_col = g.fp8_quantize(x, "row+col", stream=stream)
    if not isinstance(w, Fp8Matrix):
        w = g.fp8_quantize(w, "tile", stream=stream)
    y = g.fp8_matmul(x_row, w, bias, a_major=B.GEMM_ROW_MAJOR, b_major=B.GEMM_COL_MAJOR,
                     out_dtype=x.dtype, stream=stream)
    return y, (x_col, w)


def linear_backward(g, dy: torch.Tensor, saved, stream=None):
    """(dx, dW) of linear_forward for the gradient dy of y: dx = dy·W in dy's
    type, dW = dyᵀ·x in fp32, dy quantised along both axes in one pass."""
    x_col, w = saved
    dy_row, dy_col = g.fp8_quantize(dy, "row+col", stream=stream)
    dx = g.fp8_matmul(dy_row, w, a_major=B.GEMM_ROW_MAJOR, b_major=B.GEMM_ROW_MAJOR,
                      out_dtype=dy.dtype, stream=stream)
    dw = g.fp8_matmul(dy_col, x_col, a_major=B.GEMM_COL_MAJOR, b_major=B.GEMM_ROW_MAJOR,
                      out_dtype=torch.float32, stream=stream)
    return dx, dw


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, g, x, w, bias):
        y, ctx.saved = linear_forward(g, x, w, bias)
        ctx.g, ctx.w_dtype, ctx.has_bias = g, w.dtype, bias is not None
        return y

    @staticmethod
    def backward(ctx, dy):
        dy = dy.contiguous()
        dx, dw = linear_backward(ctx.g, dy, ctx.saved)
        return None, dx, dw.to(ctx.w_dtype), dy.float().sum(0) if ctx.has_bias else None


def linear(g, x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None = None):
    """Differentiable x·wᵀ (+bias) on handle ``g``: products in 8 bits, gradients
    passed straight through the quantisation; x (tokens, inputs) float16,
    bfloat16 or float32, w (outputs, inputs), bias float32 (outputs,)."""
    return _Linear.apply(g, x, w, bias)
