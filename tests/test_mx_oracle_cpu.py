"""The oracle of the 4-bit formats pinned by hand-computed blocks and by exact
rational arithmetic."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import admmq_oracle as O
from oracle import mx


def _exact_code(x, t):
    """e2m1 code of x / t by rational arithmetic: nearest level, ties to even."""
    u = min(Fraction(abs(float(x))) / Fraction(float(t)), Fraction(6))
    levels = [Fraction(v) for v in (0, 0.5, 1, 1.5, 2, 3, 4, 6)]
    d = [abs(u - v) for v in levels]
    best = [i for i, e in enumerate(d) if e == min(d)]
    i = best[0] if len(best) == 1 or best[0] % 2 == 0 else best[1]
    return i + (8 if np.signbit(x) else 0)


def test_hand_computed_mxfp4_block():
    """amax 7.5: e = floor(log2 7.5) - 2 = 0, so t = 1; ties 0.25, 0.75, 1.25,
    1.75, 2.5, 3.5, 5 go to the even codes, 7.5 saturates at 6."""
    x = np.zeros((1, 32), np.float32)
    x[0, :9] = [7.5, 0.25, 0.75, -1.25, 1.75, 2.5, -3.5, 5.0, 0.26]
    code, byte = mx.quantize(x, "mxfp4")
    assert byte.tolist() == [[127]]
    assert code[0, :9].tolist() == [7, 0, 2, 10, 4, 4, 14, 6, 1]
    assert mx.values(code, byte, "mxfp4")[0, :9].tolist() == [6, 0, 1, -1, 2, 2, -4, 4, 0.5]
    assert mx.quantize(np.zeros((1, 32)), "mxfp4")[1].tolist() == [[0]]
    x[0, 0] = 2.0 ** -126               # floor(log2) - 2 = -128 lies below the scale's range
    x[0, 1:] = 0
    code, byte = mx.quantize(x, "mxfp4")
    assert byte.tolist() == [[0]] and code[0, 0] == 4 and mx.values(code, byte, "mxfp4")[0, 0] == 2.0 ** -126


def test_hand_computed_nvfp4_block():
    """amax 3, g = 1: 3 / 6 = 0.5 is an e4m3 value (byte 0x30); t = 0.5."""
    x = np.zeros((1, 32), np.float32)
    x[0, :4] = [3.0, -1.25, 0.125, 0.13]     # x / t = 6, -2.5 (tie to 2), 0.25 (tie to 0), 0.26
    code, byte = mx.quantize(x, "nvfp4", 1.0)
    assert byte.tolist() == [[0x30, 0]]
    assert code[0, :4].tolist() == [7, 12, 0, 1]
    # amax / 6 below half the smallest e4m3 value: the block is zero
    x[0, :4] = 6 * 2.0 ** -11
    code, byte = mx.quantize(x, "nvfp4", 1.0)
    assert byte[0, 0] == 0 and not code.any()
    # saturated scale, saturated elements
    x[0, 0] = 1e6
    code, byte = mx.quantize(x, "nvfp4", 1.0)
    assert byte[0, 0] == 126 and code[0, 0] == 7 and mx.values(code, byte, "nvfp4", 1.0)[0, 0] == 2688


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_rounding_against_rational_arithmetic(fmt):
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((40, 64)) * np.exp(rng.uniform(-8, 8, (40, 1)))).astype(np.float32)
    g = np.float32(0.0137) if fmt == "nvfp4" else None
    code, byte = mx.quantize(x, fmt, g)
    # put elements on and next to the borders of their block's grid
    t = np.repeat(mx.step(byte, fmt, g), mx.BLOCK[fmt], axis=1)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5])
    amax = np.abs(x).reshape(40, -1, mx.BLOCK[fmt]).argmax(-1)
    for r in range(40):
        for c in range(64):
            b = c // mx.BLOCK[fmt]
            if c % mx.BLOCK[fmt] != amax[r, b] and c % 2:
                v = np.float32(rng.choice(mids) * t[r, c])
                x[r, c] = rng.choice([v, np.nextafter(v, np.float32(9e9)), np.nextafter(v, np.float32(0)), -v])
    code, byte2 = mx.quantize(x, fmt, g)
    assert np.array_equal(byte, byte2)
    want = [[_exact_code(x[r, c], t[r, c]) for c in range(64)] for r in range(40)]
    assert np.array_equal(code, want)


def test_scale_of_nvfp4_against_rational_arithmetic():
    rng = np.random.default_rng(2)
    g = np.float32(0.3)
    mids = (mx.E4M3[1:] + mx.E4M3[:-1]) / 2
    a = np.float32(mids * 6 * np.float64(g))
    x = np.zeros((3 * len(a), 16), np.float32)
    x[:, 5] = np.concatenate([a, np.nextafter(a, np.float32(0)), np.nextafter(a, np.float32(1e9))])
    _, byte = mx.quantize(x, "nvfp4", g)
    for v, b in zip(x[:, 5], byte[:, 0]):
        q = Fraction(float(v)) / (6 * Fraction(float(g)))
        d = [abs(q - Fraction(float(e))) for e in mx.E4M3]
        best = [i for i, e in enumerate(d) if e == min(d)]
        assert b == (best[0] if len(best) == 1 or best[0] % 2 == 0 else best[1])
    del rng


def test_nonfinite_blocks_read_as_nan():
    for fmt, nan in (("mxfp4", 255), ("nvfp4", 127)):
        x = np.ones((2, 64), np.float32)
        x[0, 3], x[1, 40] = np.nan, -np.inf
        code, byte = mx.quantize(x, fmt)
        v = mx.values(code, byte, fmt)
        b = mx.BLOCK[fmt]
        assert byte[0, 0] == nan and byte[1, 40 // b] == nan
        assert np.isnan(v[0, :b]).all() and np.isnan(v[1, 40 // b * b:40 // b * b + b]).all()
        assert np.isfinite(v[0, b:]).all()


def test_layouts():
    """Scale tiles by a reshape written another way; packed bits by the packing oracle."""
    rng = np.random.default_rng(3)
    byte = rng.integers(1, 200, (200, 10)).astype(np.uint8)
    full = np.zeros((256, 12), np.uint8)
    full[:200, :10] = byte
    want = full.reshape(2, 4, 32, 3, 4).transpose(0, 3, 2, 1, 4).reshape(-1)
    assert np.array_equal(mx.scale_tiles(byte), want)
    for bits in range(1, 9):
        codes = rng.integers(0, 1 << bits, (5, 96)).astype(np.uint8)
        assert np.array_equal(mx.unpack_bits(O.pack(codes, bits), bits, 96), codes)
    w = mx.packed_weights(O.pack(codes, 8), np.full((5, 3), 0.5), np.full((5, 3), 7.0), 8, 96)
    assert np.array_equal(w, 0.5 * (codes.astype(float) - 7))
    assert mx.pack_codes(np.array([[1, 15, 8, 2]], np.uint8)).tolist() == [[0xF1, 0x28]]
