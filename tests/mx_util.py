"""Microscaled 4-bit matrices in 64 bits and one value at a time where it matters: what the
GPU's codes, scales and products are held to."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127])
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def nearest(a, grid, unit):
    """Index of the grid value nearest to a / unit (a >= 0, unit > 0), ties to the even index,
    by comparing a with the midpoints times unit: products of few bits, exact in 64 bits."""
    mid = (grid[1:] + grid[:-1]) / 2
    idx = np.zeros(a.shape, np.int64)
    for i, m in enumerate(mid):
        t = m * unit
        idx += np.where(i % 2 == 0, a > t, a >= t)
    return idx


def quantize(x, fmt, g=None):
    """x (rows, cols) float -> (codes (rows, cols) 0..15, scale bytes (rows, blocks), g)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    blk = BLOCK[fmt]
    nb = -(-cols // blk)
    p = np.zeros((rows, nb * blk))
    p[:, :cols] = x
    p = p.reshape(rows, nb, blk)
    bad = ~np.isfinite(p).all(-1)
    amax = np.where(bad, 0.0, np.abs(np.where(np.isfinite(p), p, 0)).max(-1))
    if fmt == "mxfp4":
        _, e = np.frexp(amax)
        e = np.where(amax > 0, np.clip(e - 3, -127, 127), -127)
        byte, unit = e + 127, np.ldexp(1.0, e)
    else:
        if g is None:
            g = float(np.float32(np.abs(p[np.isfinite(p)]).max() / 2688.0)) or 1.0
        byte = nearest(amax, E4M3, 6 * g)
        unit = E4M3[byte] * g
    a = np.where(bad[..., None], 0.0, np.abs(np.where(np.isfinite(p), p, 0)))
    code = np.where(unit[..., None] > 0, nearest(a, GRID, unit[..., None]), 0)
    code = code + 8 * np.signbit(p)
    code = np.where(bad[..., None], 0, code)
    byte = np.where(bad, 255 if fmt == "mxfp4" else 127, byte)
    return code.reshape(rows, -1)[:, :cols], byte.astype(np.uint8), g


def scale_values(byte, fmt):
    b = byte.astype(np.int64)
    if fmt == "mxfp4":
        return np.where(b == 255, np.nan, np.ldexp(1.0, np.minimum(b, 254) - 127))
    return np.where(b == 127, np.nan, E4M3[np.minimum(b, 126)])


def values(code, byte, fmt, g=None):
    v = np.where(code >= 8, -GRID[code % 8], GRID[code % 8])
    s = np.repeat(scale_values(byte, fmt), BLOCK[fmt], axis=1)[:, :code.shape[1]]
    return v * s * (1.0 if g is None else g)


def unpack(codes, rows, cols):
    """Packed bytes of an MxTensor -> (codes (rows, cols), the row's padding codes)."""
    b = codes.reshape(rows, -1)
    c = np.stack([b & 15, b >> 4], -1).reshape(rows, -1)
    return c[:, :cols].astype(np.int64), c[:, cols:]


def untile(tiles, rows, cols, fmt):
    """The scales by the documented formula, and the bytes that belong to no block."""
    nb = -(-cols // BLOCK[fmt])
    ct = -(-nb // 4)
    r, b = np.arange(rows)[:, None], np.arange(nb)[None]
    at = 512 * (r // 128 * ct + b // 4) + 16 * (r % 32) + 4 * (r // 32 % 4) + b % 4
    rest = np.ones(tiles.size, bool)
    rest[at.reshape(-1)] = False
    return tiles[at], tiles[rest]
