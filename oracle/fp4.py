"""Microscaled 4-bit floating point and expert routing in 64 bits -- TEST INFRASTRUCTURE.

numpy, double precision, written from the definitions in include/hq.h; shares
no code with the package.  The quantiser's single-precision steps (the block
scale's quotient, the effective scale, the value's quotient) are one IEEE
rounding each: a double quotient of two fp32 numbers rounded to fp32 is the
correctly rounded fp32 quotient (53 >= 2 * 24 + 2).
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
BLOCK = {"nv": 16, "mx": 32}


def e4m3_decode(b):
    b = np.asarray(b).astype(np.int64)
    m, e = b & 7, b >> 3 & 15
    v = np.where(e > 0, (8 + m) * np.exp2(e - 10.0), m * 2.0**-9)
    return np.where((b & 127) == 127, np.nan, np.where(b & 128, -v, v))


_E4M3 = e4m3_decode(np.arange(127))


def e4m3_encode(v):
    """Nearest E4M3 byte of v >= 0, ties to the even byte, at most 448."""
    hi = np.clip(np.searchsorted(_E4M3, v), 1, 126)
    lo = hi - 1
    mid = (_E4M3[lo] + _E4M3[hi]) / 2  # exact in double
    return np.where((v > mid) | ((v == mid) & (hi % 2 == 0)), hi, lo).astype(np.uint8)


def e2m1_encode(q):
    """Nearest E2M1 code of q, ties to the even code, at most 6; the sign of q kept."""
    a = np.abs(q)
    hi = np.clip(np.searchsorted(GRID, a), 1, 7)
    lo = hi - 1
    mid = (GRID[lo] + GRID[hi]) / 2
    c = np.where((a > mid) | ((a == mid) & (hi % 2 == 0)), hi, lo)
    return (c + 8 * np.signbit(q)).astype(np.uint8)


def quantize(x, fmt, ts=None):
    """(codes [R][K] 0..15, scale bytes [R][K/block], values double [R][K]) of double rows x
    that are exact in fp32."""
    R, K = x.shape
    b = x.reshape(R, -1, BLOCK[fmt])
    fine = np.isfinite(b).all(axis=2)
    amax = np.where(fine, np.abs(np.where(np.isfinite(b), b, 0)).max(axis=2), 0)
    t = np.float64(1.0) if ts is None else np.float64(np.float32(ts))
    with np.errstate(all="ignore"):
        if fmt == "nv":
            s = e4m3_encode((amax / np.float64(np.float32(6 * t))).astype(np.float32).astype(np.float64))
            eff = (e4m3_decode(s) * t).astype(np.float32).astype(np.float64)
        else:
            _, e = np.frexp(amax)
            e = np.where(amax > 0, np.maximum(e - 3, -127), -127)
            s = (e + 127).astype(np.uint8)
            eff = np.exp2(e.astype(np.float64))
        q = np.where(eff[..., None] > 0, b / eff[..., None], np.copysign(0.0, b)).astype(np.float32).astype(np.float64)
    q = np.where(fine[..., None], q, 0.0)
    c = e2m1_encode(q)
    v = np.where(c >= 8, -1.0, 1.0) * GRID[c & 7] * eff[..., None]
    s = np.where(fine, s, 0x7F if fmt == "nv" else 0xFF).astype(np.uint8)
    v = np.where(fine[..., None], v, np.nan)
    return c.reshape(R, K), s, v.reshape(R, K)


def pack(c):
    return (c[:, ::2] | c[:, 1::2] << 4).astype(np.uint8)


def unpack(b):
    return np.stack([b & 15, b >> 4], axis=2).reshape(b.shape[0], -1)


def tile(s):
    """[R][J] scale bytes as [R/128][J/4][32][4][4] tiles, zero padded."""
    s = np.pad(s, ((0, -s.shape[0] % 128), (0, -s.shape[1] % 4)))
    return np.ascontiguousarray(s.reshape(s.shape[0] // 128, 4, 32, -1, 4).transpose(0, 3, 2, 1, 4))


def untile(t, R, J):
    return t.transpose(0, 3, 2, 1, 4).reshape(t.shape[0] * 128, -1)[:R, :J]


def values(codes, scales, fmt, ts=None):
    """double [R][K] of packed bytes [R][K/2] and scale tiles."""
    c = unpack(codes)
    R, K = c.shape
    s = untile(scales, R, K // BLOCK[fmt])
    s = e4m3_decode(s) if fmt == "nv" else np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))
    v = np.where(c >= 8, -1.0, 1.0) * GRID[c & 7]
    v = (v.reshape(R, -1, BLOCK[fmt]) * s[..., None]).reshape(R, K)
    if ts is not None:
        v = v * np.repeat(np.asarray(ts, dtype=np.float64).reshape(-1), R // np.asarray(ts).size)[:, None]
    return v


def sort(ids, E, align):
    """(pos [T][k], offsets [E + 1], counts [E]) of the stable sort by expert."""
    pos = np.full(ids.shape, -1, dtype=np.int64)
    offsets, counts, at = np.zeros(E + 1, dtype=np.int64), np.zeros(E, dtype=np.int64), 0
    flat, fp = ids.reshape(-1), pos.reshape(-1)
    for e in range(E):
        p = np.flatnonzero(flat == e)
        offsets[e], counts[e] = at, p.size
        fp[p] = at + np.arange(p.size)
        at += -(-p.size // align) * align
    offsets[E] = at
    return pos, offsets, counts
