"""4-bit microscaled matrices in plain numpy, 64 bits: the oracle of the MX tests.

Written from the format: E2M1 magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6; blocks of
32 along a row; scale 2^(byte - 127) with byte = max(0, E - 2), E the biased
fp32 exponent of the block's largest magnitude; 255 (NaN) for a block that
holds an infinity or a NaN.
"""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
#: Half-way points between neighbours of GRID, and whether a tie goes up (to the even code).
MIDS = [(0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)]


def blocks(x):
    """(rows, blocks, 32) in fp64, zeros beyond the row."""
    rows, cols = x.shape
    nb = -(-cols // 32)
    out = np.zeros((rows, nb * 32))
    out[:, :cols] = x
    return out.reshape(rows, nb, 32)


def quantize(x):
    """(codes uint8 (rows, nb, 32) , bytes (rows, nb)) of a float64 array of fp32-representable values."""
    b = blocks(np.asarray(x, dtype=np.float64))
    finite = np.isfinite(b).all(-1)
    amax = np.abs(np.where(finite[..., None], b, 0.0)).max(-1) if b.shape[-2] else np.zeros(b.shape[:2])
    _, e = np.frexp(amax)  # amax = f 2^e, 0.5 <= f < 1: exponent e - 1
    byte = np.where(amax >= 2.0 ** -126, e - 1 + 127 - 2, 0)
    byte = np.maximum(byte, 0)
    v = np.abs(np.where(finite[..., None], b, 0.0)) * 2.0 ** (127 - byte)[..., None].astype(np.float64)
    code = np.zeros(v.shape, dtype=np.uint8)
    for mid, up in MIDS:
        code += (v >= mid) if up else (v > mid)
    code |= (np.signbit(b).astype(np.uint8) << 3)
    return code, np.where(finite, byte, 255).astype(np.int64)


def values(code, byte, cols):
    """The fp64 values that codes and scale bytes stand for, cut to `cols` columns."""
    mag = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    scale = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    v = mag * scale[..., None]
    return v.reshape(v.shape[0], -1)[:, :cols]


def unpack(data, scales, rows, cols):
    """(codes, bytes) of a held matrix (numpy uint8 arrays in the library's layout)."""
    nb = -(-cols // 32)
    code = np.stack([data & 15, data >> 4], -1).reshape(rows, nb, 32)
    byte = np.zeros((rows, nb), dtype=np.int64)
    for r in range(rows):
        for b in range(nb):
            byte[r, b] = scales[r // 128, b // 4, r % 32, (r % 128) // 32 * 4 + b % 4]
    return code, byte


def same_codes(a, b):
    """Equal codes, the two zeros counted as one."""
    z = lambda c: np.where((c & 7) == 0, 0, c)  # noqa: E731
    return np.array_equal(z(a), z(b))
