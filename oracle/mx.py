"""Microscaled 4-bit floating point and the packed-code product, in float64
numpy, from their definitions (include/admmq.h states them).

Rounding is by brute force: an element (a block scale) takes the nearest level
of the whole table, ties to the even code, compared in exact rational
arithmetic where float64 could not decide (`fractions` in the tests' pins).
"""
from __future__ import annotations

import numpy as np

BLOCK = {"mxfp4": 32, "nvfp4": 16}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])  # code 127 is NaN


def nearest(u, table):
    """Index of the nearest table entry to each u >= 0, ties to the even index."""
    u = np.asarray(u, np.float64)
    d = np.abs(u[..., None] - table)
    best = d.min(-1, keepdims=True)
    hit = d == best                      # one index, or two neighbours at a tie
    first = hit.argmax(-1)
    tie = hit.sum(-1) == 2
    return np.where(tie & (first % 2 == 1), first + 1, first)


def quantize(x, fmt, g=None):
    """codes u8 [rows][k] (sign in bit 3), scale bytes u8 [rows][k / block]."""
    x = np.asarray(x, np.float64)
    rows, k = x.shape
    xb = x.reshape(rows, -1, BLOCK[fmt])
    bad = ~np.isfinite(xb).all(-1)
    xb = np.where(bad[..., None], 0.0, xb)
    amax = np.abs(xb).max(-1)
    if fmt == "mxfp4":
        with np.errstate(divide="ignore"):
            _, e = np.frexp(amax)
        e = np.where(amax > 0, np.maximum(e - 3, -127), -127)
        byte = e + 127
        t = np.ldexp(1.0, e)
    else:
        gg = 1.0 if g is None else np.float64(g)
        with np.errstate(divide="ignore", invalid="ignore"):
            q = np.where(amax > 0, np.minimum(amax / (6 * gg), 448.0), 0.0)
        byte = nearest(q, E4M3)
        t = np.float32(E4M3[byte] * gg).astype(np.float64)
    u = np.abs(xb) / np.where(t > 0, t, 1)[..., None]
    code = nearest(np.minimum(u, 6.0), E2M1)
    code = np.where((t > 0)[..., None], code + 8 * np.signbit(xb), 0)
    code = np.where(bad[..., None], 0, code)
    byte = np.where(bad, 255 if fmt == "mxfp4" else 127, byte)
    return code.reshape(rows, k).astype(np.uint8), byte.astype(np.uint8)


def step(byte, fmt, g=None):
    byte = np.asarray(byte).astype(np.int64)
    if fmt == "mxfp4":
        return np.where(byte == 255, np.nan, np.ldexp(1.0, byte - 127))
    t = np.where(byte == 127, np.nan, E4M3[np.minimum(byte, 126)])
    return np.float32(t * (1.0 if g is None else np.float64(g))).astype(np.float64)


def values(code, byte, fmt, g=None):
    code = np.asarray(code).astype(np.int64)
    v = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]
    rows, k = code.shape
    return (v.reshape(rows, -1, BLOCK[fmt]) * step(byte, fmt, g)[..., None]).reshape(rows, k)


def pack_codes(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def scale_tiles(byte):
    """Row by row, block by block, into the tiles of 512 bytes."""
    rows, blocks = byte.shape
    rt, ct = -(-rows // 128), -(-blocks // 4)
    out = np.zeros(rt * ct * 512, np.uint8)
    for r in range(rows):
        for c in range(blocks):
            q = r % 128
            out[((r // 128) * ct + c // 4) * 512 + 16 * (q % 32) + 4 * (q // 32) + c % 4] = byte[r, c]
    return out


def unpack_bits(words, bits, k):
    """Codes of packed rows: code i at bits [bits i, bits i + bits) of a row."""
    rows = words.shape[0]
    raw = np.ascontiguousarray(words).view(np.uint8).reshape(rows, -1)
    stream = np.unpackbits(raw, axis=1, bitorder="little")[:, :bits * k]
    return (stream.reshape(rows, k, bits) << np.arange(bits)).sum(-1)


def packed_weights(words, scale, zero, bits, k):
    group = k // scale.shape[1]
    c = unpack_bits(words, bits, k).astype(np.float64)
    s, z = (np.repeat(np.asarray(a, np.float64), group, axis=1) for a in (scale, zero))
    return s * (c - z)
