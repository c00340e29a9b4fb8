"""Plain numpy reference, in 64 bits, of the microscaled 4-bit (MX4) operators.

The format is MXFP4 of the OCP Microscaling Formats specification: blocks of
32 values share a power of two, the values are 4-bit floats.  Layouts follow
``include/w2a8_mx4.h`` and are written out index by index, with none of the
library's code.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def _blocks(a, K, n=32):
    """[R, K] -> [R, B, n], padded with zeros."""
    B = -(-K // n)
    out = np.zeros((a.shape[0], B * n), a.dtype)
    out[:, :K] = a
    return out.reshape(a.shape[0], B, n)


def quant(x):
    """Float rows [R, K] -> codes uint8 [R, K] (0..15) and scale bytes uint8 [R, ceil(K/32)]."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    b = _blocks(x, K)
    bad = ~np.isfinite(b).all(2)
    a = np.abs(np.where(np.isfinite(b), b, 0)).max(2)
    e = np.where(a > 0, np.frexp(a)[1] - 1 - 2, -127)      # frexp: a = f * 2^x, 1/2 <= f < 1
    e = np.maximum(e, -127)
    y = np.ldexp(np.where(bad[:, :, None], 0, b), -e[:, :, None])
    m = np.abs(y)
    # nearest of the eight magnitudes; a tie goes to the even code
    d = np.abs(m[..., None] - GRID)
    best = d.min(-1, keepdims=True)
    near = d == best
    first = near.argmax(-1)
    last = 7 - near[..., ::-1].argmax(-1)
    code = np.where(first % 2 == 0, first, last)
    code = np.where(m > 6, 7, code).astype(np.uint8)
    code |= (np.signbit(y) * 8).astype(np.uint8)
    code[bad] = 0
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    return code.reshape(R, -1)[:, :K], s


def scale_values(s):
    """Scale bytes -> powers of two in 64 bits (255: NaN)."""
    v = np.ldexp(1.0, s.astype(np.int64) - 127)
    return np.where(s == 255, np.nan, v)


def values(codes, scales):
    """Codes [R, K] and scale bytes -> float64 [R, K]."""
    v = np.concatenate([GRID, -GRID])[codes]
    return v * np.repeat(scale_values(scales), 32, axis=1)[:, :codes.shape[1]]


def _row_bytes(codes):
    """Codes [R, K] -> bytes [R, Kp / 2] in A4I order (Kp: K in whole tiles of 128)."""
    R, K = codes.shape
    Kp = -(-K // 128) * 128
    c = np.zeros((R, Kp), np.uint8)
    c[:, :K] = codes
    out = np.zeros((R, Kp // 2), np.uint8)
    for i in range(16):
        byte = 4 * (i // 4 % 2) + i % 4
        out[:, byte::8] |= c[:, i::16] << (4 if i >= 8 else 0)
    return out


def rows_layout(codes, scales):
    """MX4R: (x_q uint8 [R, 64 KT], x_s uint8 [R, 16 KU])."""
    q = _row_bytes(codes)
    R, KT = q.shape[0], q.shape[1] // 64
    KU = -(-KT // 4)
    s = np.zeros((R, 16 * KU), np.uint8)
    for b in range(scales.shape[1]):
        t, g = b // 4, b % 4
        s[:, 16 * (t // 4) + 4 * g + t % 4] = scales[:, b]
    return q, s


def packed_layout(codes, scales):
    """MX16x128 weights as one uint8 array."""
    q = _row_bytes(codes)
    N, KT = q.shape[0], q.shape[1] // 64
    KU, NS = -(-KT // 4), -(-N // 16)
    tiles = np.zeros((NS, KT, 4, 16, 16), np.uint8)         # strip, tile, block, row, byte
    sc = np.zeros((NS, KU, 4, 16, 4), np.uint8)             # strip, four tiles, block, row, tile
    s, r = np.arange(N) // 16, np.arange(N) % 16
    tiles[s, :, :, r, :] = q.reshape(N, KT, 4, 16)
    for b in range(scales.shape[1]):
        t, g = b // 4, b % 4
        sc[s, t // 4, g, r, t % 4] = scales[:, b]
    return np.concatenate([tiles.reshape(-1), sc.reshape(-1)])


def interchange(codes):
    """Codes [R, K] two a byte, the lower k in the lower half: uint8 [R, ceil(K/2)]."""
    R, K = codes.shape
    c = np.zeros((R, K + K % 2), np.uint8)
    c[:, :K] = codes
    return c[:, 0::2] | (c[:, 1::2] << 4)


def product(x, w, s_w=1.0):
    """Float64 rows [M, K] times weights [N, K]: (y [M, N], sum of magnitudes [M, N])."""
    with np.errstate(invalid="ignore"):
        return (x @ w.T) * s_w, (np.abs(x) @ np.abs(w).T) * abs(s_w)
