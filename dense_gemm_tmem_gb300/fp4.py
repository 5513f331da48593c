"""4-bit matrices and the linear layer served with them.

``Fp4Matrix`` holds what `Gemm.fp4_quantize` writes and `Gemm.fp4_matmul` and
`Gemm.fp4_dequantize` read: e2m1 values, two to a byte, with a scale for each block
of neighbours along a row.  ``"mxfp4"`` has blocks of 32 with power-of-two scales,
``"nvfp4"`` blocks of 16 with e4m3 scales and one fp32 scale per row.  ``linear`` is a
linear layer on a weight stored so.
"""
from __future__ import annotations

import torch

from . import binding as B

FORMATS = {"mxfp4": B.GEMM_MXFP4, "nvfp4": B.GEMM_NVFP4}
BLOCK = {"mxfp4": 32, "nvfp4": 16}
_BYTES = (torch.uint8, getattr(torch, "float4_e2m1fn_x2", torch.uint8))
_SCALES = {"mxfp4": (torch.uint8, getattr(torch, "float8_e8m0fnu", torch.uint8)),
           "nvfp4": (torch.uint8, torch.float8_e4m3fn)}
_new = object.__new__


def _format(name: str) -> int:
    code = FORMATS.get(name)
    if code is None:
        raise ValueError("format must be 'mxfp4' or 'nvfp4', got %r" % (name,))
    return code


def scale_bytes(rows: int, cols: int, format: str) -> int:
    """Bytes of the block scales: whole pieces of 128 rows x 4 blocks."""
    _format(format)
    return (rows + 127) // 128 * (-(-cols // (4 * BLOCK[format]))) * 512


def pack_scales(scale: torch.Tensor) -> torch.Tensor:
    """Block scales (rows, blocks; one byte each) in the order they are stored in
    (include/gemm_fp4.h), bytes past the matrix 0."""
    r, b = scale.shape
    s = scale.view(torch.uint8)
    out = s.new_zeros((-(-r // 128)) * 128, -(-b // 4) * 4)
    out[:r, :b] = s
    return out.view(-(-r // 128), 4, 32, -(-b // 4), 4).permute(0, 3, 2, 1, 4).reshape(-1)


def unpack_scales(scale: torch.Tensor, rows: int, blocks: int) -> torch.Tensor:
    """The (rows, blocks) bytes of stored block scales."""
    s = scale.view(torch.uint8).view(-(-rows // 128), -(-blocks // 4), 32, 4, 4)
    return s.permute(0, 3, 2, 1, 4).reshape(-(-rows // 128) * 128, -1)[:rows, :blocks]


def _check(data, scale, row_scale, rows, cols, format):
    """Refuses what is no 4-bit matrix."""
    if data.dtype not in _BYTES:
        raise TypeError("data must be uint8 (or float4_e2m1fn_x2), got %s" % data.dtype)
    if scale.dtype not in _SCALES[format]:
        raise TypeError("scale must be uint8 or the format's scale type, got %s" % scale.dtype)
    if rows < 0 or cols < 0 or data.shape != (rows, (cols + 1) // 2):
        raise ValueError("data has shape %s, expected (%d, %d)"
                         % (tuple(data.shape), rows, (cols + 1) // 2))
    st = data.stride()
    if (data.shape[1] > 1 and st[1] != 1) or (rows > 1 and st[0] < data.shape[1]):
        raise ValueError("rows of data must be contiguous and not overlap")
    if scale.dim() != 1 or scale.shape[0] != scale_bytes(rows, cols, format) or (
            scale.shape[0] > 1 and scale.stride(0) != 1):
        raise ValueError("scale must be contiguous and flat, of %d bytes"
                         % scale_bytes(rows, cols, format))
    if row_scale is not None:
        if row_scale.dtype != torch.float32:
            raise TypeError("row_scale must be float32, got %s" % row_scale.dtype)
        if row_scale.shape != (rows,):
            raise ValueError("row_scale has shape %s, expected (%d,)"
                             % (tuple(row_scale.shape), rows))
    for t in (scale, row_scale):
        if t is not None and t.get_device() != data.get_device():
            raise ValueError("data on %s, scales on %s" % (data.device, t.device))


class Fp4Matrix:
    """A (rows, cols) matrix in 4 bits.  ``data`` (rows, ceil(cols / 2)) has the even
    column in the low half of each byte, unit stride along its rows, which start on
    16 bytes (rows padded to 16, as ``fp4_quantize`` pads them); the high half of an
    odd row's last byte is 0.  ``scale`` is the flat tensor of block scales in their
    stored order (see ``pack_scales``), nvfp4's with no sign bit set, ``row_scale`` None or float32 (rows,), of any
    stride (``scale.expand(rows)`` for one scale of the whole matrix).  The tensors
    are referenced, not copied; replacing them in place is seen by later calls."""

    __slots__ = ("data", "scale", "row_scale", "shape", "format", "kind")

    def __init__(self, data: torch.Tensor, scale: torch.Tensor, row_scale, shape, format: str):
        rows, cols = shape
        kind = FORMATS.get(format)
        if kind is None:
            _format(format)
        # the extension's checks where it is loaded (0.5 us of a decode step's time, not 2)
        if B._native is not None:
            B._native.check4(data, scale, row_scale, rows, cols, kind)
        else:
            _check(data, scale, row_scale, rows, cols, format)
        self.data, self.scale, self.row_scale = data, scale, row_scale
        self.shape, self.format, self.kind = (rows, cols), format, kind

    @staticmethod
    def _wrap(data, scale, row_scale, shape, format):
        """What the quantiser made, without checks."""
        m = _new(Fp4Matrix)
        m.data, m.scale, m.row_scale = data, scale, row_scale
        m.shape, m.format, m.kind = shape, format, FORMATS[format]
        return m

    @staticmethod
    def from_parts(data: torch.Tensor, scale: torch.Tensor, row_scale=None, cols: int = None,
                   format: str = "nvfp4") -> "Fp4Matrix":
        """From packed values (rows, ceil(cols / 2)) and block scales (rows, blocks) as
        checkpoints hold them; row_scale float32, one for the matrix or one per row.
        Laid out anew: rows on 16 bytes, scales in their stored order."""
        _format(format)
        rows, width = data.shape
        cols = 2 * width if cols is None else int(cols)
        blocks = -(-cols // BLOCK[format])
        if width != (cols + 1) // 2 or tuple(scale.shape) != (rows, blocks):
            raise ValueError("data has shape %s and scale %s, expected (rows, %d) and (rows, %d)"
                             % (tuple(data.shape), tuple(scale.shape), (cols + 1) // 2, blocks))
        if scale.dtype not in _SCALES[format]:
            raise TypeError("scale must be uint8 or the format's scale type, got %s"
                            % scale.dtype)
        buf = torch.zeros((rows, (width + 15) & -16), dtype=torch.uint8, device=data.device)
        buf[:, :width] = data.view(torch.uint8)
        if cols % 2:
            buf[:, width - 1] &= 15
        if row_scale is not None:
            row_scale = row_scale.reshape(-1).expand(rows)
        return Fp4Matrix(buf[:, :width], pack_scales(scale), row_scale, (rows, cols), format)

    def block_scales(self) -> torch.Tensor:
        """The block scales' bytes, (rows, blocks)."""
        return unpack_scales(self.scale, self.shape[0], -(-self.shape[1] // BLOCK[self.format]))

    def desc(self) -> "B.gemm_fp4_matrix_t":
        """The C-ABI's description."""
        rows, width = self.data.shape
        ld = self.data.stride(0) if rows > 1 else (width + 15) & -16
        r = self.row_scale
        return B.gemm_fp4_matrix_t(self.data.data_ptr(), ld, self.scale.data_ptr(),
                                   None if r is None else r.data_ptr(),
                                   0 if r is None else r.stride(0), self.kind, 0)


def linear(g, x: torch.Tensor, w: Fp4Matrix, bias: torch.Tensor | None = None, stream=None):
    """x·wᵀ (+bias) in x's type on handle ``g``, x (tokens, inputs) float16, bfloat16 or
    float32 quantised to w's format row by row (what a token is quantised to does not
    depend on the others; its sums are made in an order that depends on how many there
    are, so that their last fp32 bits may), w an Fp4Matrix (outputs, inputs), bias
    float32 (outputs,).  It carries no gradient.  With a stream: as `Gemm.fp4_matmul`."""
    return g.fp4_linear(x, w, bias, stream)
