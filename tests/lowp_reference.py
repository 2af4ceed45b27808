"""Plain 64-bit forms of the low-precision operators, for the tests: numpy,
written from the formats' definitions."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m / 512.0 for m in range(8)] +
                [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)])[:127]  # byte 0x7F is NaN
BLOCK = {"nvfp4": 16, "mxfp4": 32}


def kpad(K):
    return -(-K // 64) * 64


def nearest(grid, q):
    """Index of the grid value nearest to q >= 0, of two equally near ones the even index; the last beyond the end."""
    up = np.clip(np.searchsorted(grid, q), 1, len(grid) - 1)
    lo, hi = q - grid[up - 1], grid[up] - q
    return np.where((lo < hi) | ((lo == hi) & (up % 2 == 1)), up - 1, up)


def quantize(x, fmt, prescale=1.0):
    """(codes [rows, kpad], scale bytes [rows, blocks]) of the rows of x."""
    with np.errstate(over="ignore", invalid="ignore"):
        x = (x.astype(np.float32) * np.float32(prescale)).astype(np.float64)
    rows, K = x.shape
    blk = BLOCK[fmt]
    v = np.zeros((rows, kpad(K)))
    v[:, :K] = x
    v = v.reshape(rows, -1, blk)
    finite = np.isfinite(v).all(axis=2)
    v = np.where(finite[..., None], v, 0.0)
    top = np.abs(v).max(axis=2)
    if fmt == "mxfp4":
        _, e = np.frexp(top)
        byte = np.where(top > 0, np.clip(e - 3, -127, 127) + 127, 0)
        scale = np.where(top > 0, np.ldexp(1.0, byte - 127), 0.0)
        nan = 0xFF
    else:
        byte = nearest(E4M3, top / 6.0)
        scale = E4M3[byte]
        nan = 0x7F
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(scale[..., None] > 0, np.abs(v) / scale[..., None], 0.0)
    code = nearest(E2M1, q)
    code = np.where(finite[..., None], code, 0)
    neg = np.signbit(v) & finite[..., None]
    return code.reshape(rows, -1), neg.reshape(rows, -1), np.where(finite, byte, nan).astype(np.uint8)


def scale_values(byte, fmt):
    byte = byte.astype(np.int64)
    if fmt == "mxfp4":
        return np.where(byte == 255, np.nan, np.ldexp(1.0, byte - 127))
    return np.where(byte == 127, np.nan, E4M3[np.minimum(byte, 126)])


def values(code, neg, byte, fmt, K):
    s = np.repeat(scale_values(byte, fmt), BLOCK[fmt], axis=1)
    return (np.where(neg, -1.0, 1.0) * E2M1[code] * s)[:, :K]


def stored_codes(codes, K):
    """(code, sign) of stored code bytes [rows, kpad / 2]."""
    both = np.stack((codes & 15, codes >> 4), axis=2).reshape(codes.shape[0], -1)
    return both & 7, both >= 8


def stored_scales(scales, rows, K, fmt, starts):
    """Scale bytes [rows, blocks] out of the tiles; starts: group starts (and the end)."""
    blocks = kpad(K) // BLOCK[fmt]
    tiles = -(-blocks // 4)
    out = np.zeros((rows, blocks), dtype=np.uint8)
    b = np.arange(blocks)
    for g in range(len(starts) - 1):
        for row in range(starts[g], starts[g + 1]):
            r = row - starts[g]
            at = ((starts[g] // 128 + g + r // 128) * tiles + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4
            out[row] = scales[at]
    return out


def grouped(x, w, starts):
    return np.concatenate([x[a:b] @ w[g].T for g, (a, b) in enumerate(zip(starts[:-1], starts[1:]))])


def grouped_dx(dy, w, starts):
    return np.concatenate([dy[a:b] @ w[g] for g, (a, b) in enumerate(zip(starts[:-1], starts[1:]))])


def grouped_dw(dy, x, starts):
    return np.stack([dy[a:b].T @ x[a:b] for a, b in zip(starts[:-1], starts[1:])])
