"""fp64 oracle of the microscaled formats, their product and the residual
RMSNorm.  Blocks of 32 columns; the scale is the smallest 2^k with
max|v| <= 2^k * (largest code), clamped to k in [-127, 127] (-127 for zeros);
codes are nearest to v / 2^k, ties to the even code.  Shares no code with the
CUDA path: values are placed by search in the formats' value tables."""
from __future__ import annotations

import numpy as np

GRID4 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
GRID8 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
                  for e in range(16) for m in range(8) if not (e == 15 and m == 7)], dtype=np.float64)


def up(n: int, m: int) -> int:
    return (n + m - 1) // m * m


def scale_exponents(v, top: float):
    """k per (row, block) of a [rows, cols] matrix; NaN blocks give 128."""
    rows, cols = v.shape
    b = np.zeros((rows, up(cols, 32)))
    b[:, :cols] = v
    b = b.reshape(rows, -1, 32)
    bad = ~np.isfinite(b).all(-1)
    amax = np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0)).max(-1))
    k = np.full(amax.shape, -127, dtype=np.int64)
    for i, a in np.ndenumerate(amax):
        if a > 0:
            e = int(np.floor(np.log2(a / top))) - 1
            while a > top * 2.0 ** e:
                e += 1
            k[i] = min(max(e, -127), 127)
    k[bad] = 128
    return k


def quantize(v, grid):
    """(codes [rows, cols] with the sign in the bit above the grid, k)."""
    v = np.asarray(v, dtype=np.float64)
    rows, cols = v.shape
    k = scale_exponents(v, grid[-1])
    kk = np.repeat(k, 32, axis=1)[:, :cols]
    bad = kk == 128
    a = np.abs(np.where(bad, 0.0, v)) / 2.0 ** np.where(bad, 0, kk)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo_d, hi_d = a - grid[hi - 1], grid[hi] - a
    code = np.where((hi_d < lo_d) | ((hi_d == lo_d) & (hi % 2 == 0)), hi, hi - 1)
    top = 8 if len(grid) == 8 else 128
    return np.where(bad, 0, code + np.where(np.signbit(v), top, 0)).astype(np.uint8), k


def values(codes, k, grid):
    top = 8 if len(grid) == 8 else 128
    c = codes.astype(np.int64)
    v = grid[np.minimum(c % top, len(grid) - 1)] * np.where(c >= top, -1.0, 1.0)
    kk = np.repeat(k, 32, axis=1)[:, :codes.shape[1]]
    return np.where(kk == 128, np.nan, v * 2.0 ** np.where(kk == 128, 0, kk))


def layout(rows: int, cols: int, mx4: bool) -> dict:
    rp, cp = up(rows, 128), up(cols, 128)
    q = rp * cp // 2 if mx4 else rows * cp
    s = up(q, 256)
    return {"cols_padded": cp, "q_bytes": q, "s_offset": s, "s_bytes": rp * cp // 32, "total": up(s + rp * cp // 32, 256)}


def scale_places(rows: int, cols: int):
    """Byte of every (row, block) in the scale section, padded blocks included."""
    nt = up(cols, 128) // 128
    r = np.arange(rows)[:, None]
    b = np.arange(nt * 4)[None, :]
    return ((r // 128) * nt + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4


def pack4(codes, k):
    """The packed bytes of an MXFP4 matrix (padding: code 0, scale byte 0)."""
    rows, cols = codes.shape
    L = layout(rows, cols, True)
    buf = np.zeros(L["total"], dtype=np.uint8)
    nt = L["cols_padded"] // 128
    r = np.arange(rows)[:, None]
    c = np.arange(cols)[None, :]
    np.bitwise_or.at(buf, ((r // 128) * nt + c // 128) * 8192 + (r % 128) * 64 + (c % 128) // 2,
                     (codes << (4 * (c % 2))).astype(np.uint8))
    kb = np.zeros((rows, nt * 4), dtype=np.uint8)
    kb[:, :k.shape[1]] = (k + 127).astype(np.uint8)
    buf[L["s_offset"] + scale_places(rows, cols)] = kb
    return buf


def unpack8(buf, tokens: int, cols: int):
    """(codes, k) of packed MXFP8 tokens."""
    L = layout(tokens, cols, False)
    codes = buf[:L["q_bytes"]].reshape(tokens, -1)
    k = buf[L["s_offset"] + scale_places(tokens, cols)].astype(np.int64) - 127
    return codes, k


def rmsnorm(x, residual=None, weight=None, eps=1e-6):
    """(h, y) in fp64."""
    h = np.asarray(x, dtype=np.float64) + (0.0 if residual is None else np.asarray(residual, dtype=np.float64))
    y = h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps)
    return h, y if weight is None else y * np.asarray(weight, dtype=np.float64)
