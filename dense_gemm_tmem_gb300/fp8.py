"""Block-scaled 8-bit matrices and the layers built on them.

``Fp8Matrix`` holds what `Gemm.fp8_quantize` writes and `Gemm.fp8_matmul` and
`Gemm.moe_fp8` read: e4m3 values with one fp32 scale for each block of 128
(``"row"`` 1 x 128, ``"col"`` 128 x 1, ``"tile"`` 128 x 128).  ``linear_forward``
and ``linear_backward`` are the three products of a linear layer on them, and
``linear`` the same as a differentiable function.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding as B

BLOCK = 128
BLOCKS = {"row": B.GEMM_FP8_ROW, "col": B.GEMM_FP8_COL, "tile": B.GEMM_FP8_TILE}
_BYTES = (torch.float8_e4m3fn, torch.uint8)
_new = object.__new__


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

    __slots__ = ("data", "scale", "blocks", "kind")

    def __init__(self, data: torch.Tensor, scale: torch.Tensor, blocks: str):
        if data.dtype not in _BYTES:
            raise TypeError("data must be float8_e4m3fn (or its bytes as uint8), got %s"
                            % data.dtype)
        if scale.dtype != torch.float32:
            raise TypeError("scale must be float32, got %s" % scale.dtype)
        shape = data.shape
        if len(shape) not in (2, 3):
            raise ValueError("data must be 2-D, or 3-D with one matrix per expert")
        rows, cols = shape[-2:]
        st = data.stride()
        if (cols > 1 and st[-1] != 1) or (rows > 1 and st[-2] < cols):
            raise ValueError("rows of data must be contiguous and not overlap")
        want = scale_shape(rows, cols, blocks)
        if len(shape) == 3:
            if blocks != "tile":
                raise ValueError("expert weights have tile blocks")
            want = (shape[0],) + want
        if scale.shape != want:
            raise ValueError("scale has shape %s, expected %s" % (tuple(scale.shape), want))
        if scale.get_device() != data.get_device():
            raise ValueError("data on %s, scale on %s" % (data.device, scale.device))
        self.data, self.scale, self.blocks, self.kind = data, scale, blocks, BLOCKS[blocks]

    @staticmethod
    def empty(rows: int, cols: int, blocks: str, device) -> "Fp8Matrix":
        """Unwritten storage as fp8_quantize lays it: rows padded to 16 bytes;
        the scales of 1 x 128 blocks with those of one k-block next to each
        other (the order the product's threads read them in), others row-major."""
        data = torch.empty((rows, (cols + 15) & -16), dtype=torch.float8_e4m3fn, device=device)
        shape = scale_shape(rows, cols, blocks)
        if blocks == "row":
            scale = torch.empty(shape[::-1], dtype=torch.float32, device=device).t()
        else:
            scale = torch.empty(shape, dtype=torch.float32, device=device)
        return Fp8Matrix(data[:, :cols], scale, blocks)

    @staticmethod
    def _wrap(data, scale, blocks):
        """What the quantiser made, without checks."""
        m = _new(Fp8Matrix)
        m.data, m.scale, m.blocks, m.kind = data, scale, blocks, BLOCKS[blocks]
        return m

    @property
    def shape(self):
        return self.data.shape

    def desc(self) -> "B.gemm_fp8_matrix_t":
        """The C-ABI's description of a 2-D matrix."""
        rows, cols = self.data.shape
        sr, sc = self.scale.stride()
        ld = self.data.stride(0)
        return B.gemm_fp8_matrix_t(self.data.data_ptr(), ld if rows > 1 else max(ld, cols),
                                   self.scale.data_ptr(), sr, sc, self.kind, 0)

    def dequantize(self) -> torch.Tensor:
        """fp32 values, in plain torch (for checks and small matrices)."""
        r, c = self.data.shape[-2:]
        s = self.scale
        if self.blocks != "row":
            s = s.repeat_interleave(BLOCK, -2)[..., :r, :]
        if self.blocks != "col":
            s = s.repeat_interleave(BLOCK, -1)[..., :c]
        return self.data.view(torch.float8_e4m3fn).float() * s


def linear_forward(g, x: torch.Tensor, w, bias: torch.Tensor | None = None, stream=None,
                   need_dw: bool = True):
    """y = x·Wᵀ (+bias) in 8 bits, and what linear_backward needs: x (tokens,
    inputs) is quantised along both axes in one pass (along its rows only when
    no dW is needed), w is (outputs, inputs) or an Fp8Matrix of it with tile
    blocks.  y has x's type."""
    if need_dw:
        x_row, x_col = g.fp8_quantize(x, "row+col", stream=stream)
    else:
        x_row, x_col = g.fp8_quantize(x, "row", stream=stream), None
    if not isinstance(w, Fp8Matrix):
        w = g.fp8_quantize(w, "tile", stream=stream)
    y = g.fp8_matmul(x_row, w, bias, a_major=B.GEMM_ROW_MAJOR, b_major=B.GEMM_COL_MAJOR,
                     out_dtype=x.dtype, stream=stream)
    return y, (x_col, w)


def linear_backward(g, dy: torch.Tensor, saved, stream=None, need_dx: bool = True,
                    need_dw: bool = True, dw_dtype=torch.float32):
    """(dx, dW) of linear_forward for the gradient dy of y: dx = dy·W in dy's
    type, dW = dyᵀ·x summed in fp32 and rounded once to dw_dtype, dy quantised
    along both axes in one pass.  One that is not needed is None and costs
    nothing."""
    x_col, w = saved
    if need_dw and x_col is None:
        raise ValueError("linear_forward was told that no dW is needed")
    dx = dw = dy_row = dy_col = None
    if need_dx and need_dw:
        dy_row, dy_col = g.fp8_quantize(dy, "row+col", stream=stream)
    elif need_dx:
        dy_row = g.fp8_quantize(dy, "row", stream=stream)
    elif need_dw:
        dy_col = g.fp8_quantize(dy, "col", stream=stream)
    if need_dx:
        dx = g.fp8_matmul(dy_row, w, a_major=B.GEMM_ROW_MAJOR, b_major=B.GEMM_ROW_MAJOR,
                          out_dtype=dy.dtype, stream=stream)
    if need_dw:
        dw = g.fp8_matmul(dy_col, x_col, a_major=B.GEMM_COL_MAJOR, b_major=B.GEMM_ROW_MAJOR,
                          out_dtype=dw_dtype, stream=stream)
    return dx, dw


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, g, x, w, bias, need_dx, need_dw):
        y, (x_col, wq) = linear_forward(g, x, w, bias, need_dw=need_dw)
        ctx.save_for_backward(*((x_col.data, x_col.scale) if need_dw else (None, None)),
                              *((wq.data, wq.scale) if need_dx else (None, None)))
        ctx.g, ctx.w_dtype, ctx.need = g, w.dtype, (need_dx, need_dw)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        need_dx, need_dw = ctx.need
        x_data, x_scale, w_data, w_scale = ctx.saved_tensors
        dx = dw = None
        if need_dx or need_dw:
            dy = dy.contiguous()
            saved = (Fp8Matrix._wrap(x_data, x_scale, "col") if need_dw else None,
                     Fp8Matrix._wrap(w_data, w_scale, "tile") if need_dx else None)
            dx, dw = linear_backward(ctx.g, dy, saved, need_dx=need_dx, need_dw=need_dw,
                                     dw_dtype=ctx.w_dtype)
        dbias = dy.sum(0, dtype=torch.float32) if ctx.needs_input_grad[3] else None
        return None, dx, dw, dbias, None, None


def linear(g, x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None = None):
    """Differentiable x·wᵀ (+bias) on handle ``g``: products in 8 bits, gradients
    passed straight through the quantisation; x (tokens, inputs) float16,
    bfloat16 or float32, w (outputs, inputs), bias float32 (outputs,).  What
    needs no gradient is neither kept nor computed."""
    grad = torch.is_grad_enabled()
    return _Linear.apply(g, x, w, bias, grad and x.requires_grad, grad and w.requires_grad)
