"""The 4-bit formats in plain numpy doubles, from their definition."""
import numpy as np

BLOCK = {"mxfp4": 32, "nvfp4": 16}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def f32(v):
    """Doubles rounded to fp32 (subnormals kept), as doubles."""
    with np.errstate(over="ignore"):
        return np.asarray(v).astype(np.float32).astype(np.float64)


def round_e2m1(v):
    """Codes of the nearest e2m1 values, ties to the even code."""
    a = np.abs(v)
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    code = np.zeros(a.shape, np.int64)
    for i, m in enumerate(mid):  # code i + 1 from the middle on, or beyond it
        code += (a >= m) if (i + 1) % 2 == 0 else (a > m)
    return code + 8 * np.signbit(v)


def e4m3(byte):
    byte = np.asarray(byte).astype(np.int64)
    e, m = (byte >> 3) & 15, byte & 7
    v = np.where(e > 0, (8.0 + m) * np.exp2(e - 10.0), m * 2.0 ** -9)
    return np.where((byte & 127) == 127, np.nan, np.where(byte & 128, -v, v))


def to_e4m3(v):
    """Bytes of the nearest e4m3 values of non-negative doubles up to 448 (and a bit)."""
    table = e4m3(np.arange(127))
    mid = (table[1:] + table[:-1]) / 2
    lo = np.searchsorted(mid, v, side="left")    # ties down
    hi = np.searchsorted(mid, v, side="right")   # ties up
    return np.where(lo % 2 == 0, lo, hi).astype(np.uint8)


def scale_value(byte, fmt):
    if fmt == "nvfp4":
        return e4m3(byte)
    b = np.asarray(byte).astype(np.float64)
    return np.where(b == 255, np.nan, np.exp2(b - 127))


def quantize(x, fmt):
    """(codes rows x cols, scale bytes rows x blocks, row scales or None) of doubles."""
    n = BLOCK[fmt]
    r, c = x.shape
    nb = -(-c // n)
    p = np.zeros((r, nb * n))
    p[:, :c] = x
    p = p.reshape(r, nb, n)
    fine = np.isfinite(p)
    a = np.where(fine, np.abs(p), 0.0)
    amax = a.max(2)
    odd = ~fine.all(2)
    if fmt == "mxfp4":
        with np.errstate(divide="ignore"):
            e = np.clip(np.floor(np.log2(np.maximum(amax, 2.0 ** -149))) - 2, -127, 127)
        # log2 of doubles may round up to a power of two that amax does not reach
        e = np.where(np.exp2(e + 2) > np.maximum(amax, 2.0 ** -125), np.maximum(e - 1, -127), e)
        byte = (e + 127).astype(np.uint8)
        factor = np.exp2(-e)
        code = round_e2m1(np.where(odd[..., None], 0.0, np.where(fine, p, 0) * factor[..., None]))
        byte = np.where(odd, 255, byte).astype(np.uint8)
        rows = None
    else:
        top = np.maximum(amax.max(1), 2.0 ** -100)[:, None]
        byte = to_e4m3(f32(amax * f32(448.0 / top)))
        s = e4m3(byte)
        k = np.where(s > 0, f32(f32(2688.0 / top) / np.where(s > 0, s, 1)), 0.0)
        code = round_e2m1(np.where(odd[..., None], 0.0, f32(np.where(fine, p, 0) * k[..., None])))
        byte = np.where(odd, 0x7f, byte).astype(np.uint8)
        rows = f32(top / 2688.0)[:, 0]
    return code.reshape(r, -1)[:, :c], byte, rows


def times_blocks(code, byte, fmt):
    """value * block scale of every element."""
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.repeat(scale_value(byte, fmt), BLOCK[fmt], 1)[:, :code.shape[1]]
    return v * s


def pack(code):
    r, c = code.shape
    p = np.zeros((r, c + c % 2), np.int64)
    p[:, :c] = code
    return (p[:, ::2] + 16 * p[:, 1::2]).astype(np.uint8)


def unpack(data, cols):
    return np.stack((data & 15, data >> 4), 2).reshape(data.shape[0], -1)[:, :cols].astype(np.int64)


def place(r, b, blocks):
    """Where the scale of row r, block b is stored."""
    return ((r // 128) * -(-blocks // 4) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4


def stored(m):
    """(codes, scale bytes rows x blocks) of an Fp4Matrix, read by the documented places."""
    rows, cols = m.shape
    blocks = -(-cols // BLOCK[m.format])
    code = unpack(m.data.cpu().numpy(), cols)
    r, b = np.arange(rows)[:, None], np.arange(blocks)[None, :]
    return code, m.scale.cpu().numpy()[place(r, b, blocks)]


def values(m):
    """What an Fp4Matrix stands for, in doubles."""
    code, byte = stored(m)
    v = times_blocks(code, byte, m.format)
    return v if m.row_scale is None else v * m.row_scale.double().cpu().numpy()[:, None]
