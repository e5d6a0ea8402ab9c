"""Pins of the CPU oracle for the four-bit formats (no GPU): the formats' values
against torch's, roundings against exact rational arithmetic, scales, ties, values
that are not finite, the packed layout, and the block's forward against its plain
formula where quantisation loses nothing."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import fp4 as O
from oracle import mlp as OM


def rng(seed):
    return np.random.default_rng(seed)


def test_e4m3_values_are_torchs():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    assert np.array_equal(O.E4M3, t.numpy())


def nearest(value, table):
    """The code of the nearest table value to a Fraction, ties to the even one."""
    best = min(abs(value - Fraction(t)) for t in table)
    hits = [i for i, t in enumerate(table) if abs(value - Fraction(t)) == best]
    return next((i for i in hits if i % 2 == 0), hits[0])


def test_e4m3_rounding_is_the_nearest_value():
    mids = (O.E4M3[1:] + O.E4M3[:-1]) / 2
    x = np.concatenate([mids, np.nextafter(mids, 0), np.nextafter(mids, 1e9),
                        rng(0).uniform(0, 500, 200), [0, 448, 449, 1e9]])
    got = O.round_e4m3(x)
    for v, c in zip(x, got):
        assert c == nearest(Fraction(float(v)), O.E4M3), v
    # a quotient that is not a number of 53 bits: compared before dividing
    for num in (1.0, 10.0, 0.1, 7 * 2.0 ** -8):
        for den in (6.0, 6.0 * 2 ** -20):
            want = nearest(Fraction(num) / Fraction(den), O.E4M3)
            assert O.round_e4m3(np.array([num]), den)[0] == want


def test_e2m1_rounding_is_the_nearest_value():
    for unit in (1.0, 0.875, 13 * 2.0 ** -4, 448.0, 2.0 ** -9):
        mids = (O.E2M1[1:] + O.E2M1[:-1]) / 2 * unit
        x = np.concatenate([mids, np.nextafter(mids, 0), np.nextafter(mids, 1e9),
                            rng(1).uniform(0, 7, 100) * unit, [0, 100 * unit]])
        got = O.round_e2m1(x, np.full(x.shape, unit))
        for v, c in zip(x, got):
            assert c == nearest(Fraction(float(v)) / Fraction(unit), O.E2M1), v
    assert (O.round_e2m1(np.ones(3), np.zeros(3)) == 0).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_what_the_format_holds_is_kept(fmt):
    """Codes times scales, quantised again, are themselves."""
    r = rng(2)
    size = O.BLOCK[fmt]
    codes = r.integers(0, 16, (5, 4 * size))
    codes[:, ::size] = 7                 # every block's largest is 6
    if fmt == "mxfp4":
        byte = r.integers(100, 150, (5, 4))
        g = 1.0
    else:
        byte = r.integers(8, 127, (5, 4))
        byte[0, 0] = 126
        g = 2.0 ** -5
    x = O.values(codes, byte, g, fmt)
    c2, b2, g2 = O.quantize(x, fmt)
    assert g2 == g and np.array_equal(b2, byte)
    assert np.array_equal(O.values(c2, b2, g2, fmt), x)
    assert np.array_equal(c2 & 7, codes & 7)


def test_mx_scale_is_two_below_the_largest_exponent():
    for top in (1.0, 1.99, 2.0, 5.0, 6.0, 7.9, 8.0, 3e38, 2.0 ** -126, 2.0 ** -140):
        x = np.zeros((1, 32))
        x[0, 5] = -top
        c, b, _ = O.quantize(x, "mxfp4")
        e = max(math.floor(math.log2(top)) - 2, -127)
        assert b[0, 0] == e + 127
        q = min(top / 2.0 ** e, 6.0)
        assert O.E2M1[c[0, 5] & 7] == O.E2M1[nearest(Fraction(q), O.E2M1)]
    c, b, _ = O.quantize(np.zeros((1, 40)), "mxfp4")
    assert (b == 127).all() and (c == 0).all()


def test_nv_scale_of_the_matrix():
    assert O.auto_scale(np.zeros((2, 2))) == 1.0
    assert O.auto_scale([2688.0]) == 1.0
    assert O.auto_scale([np.nextafter(2688.0, 1e9)]) == 2.0
    assert O.auto_scale([1344.0, np.inf, np.nan]) == 0.5
    assert O.auto_scale([1e-44]) == 2.0 ** -126
    x = rng(3).normal(size=(3, 50))
    c, b, g = O.quantize(x, "nvfp4")
    assert np.abs(x).max() <= 2688 * g and np.abs(x).max() > 1344 * g
    assert b.max() <= 126 and b.max() >= 119     # 224 .. 448


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_a_block_with_a_value_that_is_not_finite_is_nan(fmt):
    size = O.BLOCK[fmt]
    x = rng(4).normal(size=(2, 3 * size))
    x[0, size] = np.inf
    x[1, 2 * size + 3] = np.nan
    v = O.quantized(x, fmt)
    want = np.zeros(x.shape, dtype=bool)
    want[0, size:2 * size] = True
    want[1, 2 * size:] = True
    assert np.array_equal(np.isnan(v), want)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_error_is_half_a_step(fmt):
    """Against the block's scale, an element is off by half the step of its
    binade, or by what lies above 6 (NV: a scale rounded down by at most 1/16; MX:
    a largest quotient below 8)."""
    x = rng(5).normal(size=(64, 64)) * 10
    c, b, g = O.quantize(x, fmt, 1.0)
    s = np.repeat(O.scale_values(b, fmt), O.BLOCK[fmt], 1) * g
    q, v = np.abs(x) / s, O.E2M1[c & 7]
    step = np.where(q < 2, 0.25, np.where(q < 4, 0.5, 1.0))
    over = 6 / 16 if fmt == "nvfp4" else 2.0
    assert (np.abs(q - v) <= np.where(q > 6, over, step)).all()


def test_packed_layout_by_hand():
    codes = np.zeros((130, 257), dtype=np.int64)
    byte = np.zeros((130, 17), dtype=np.int64)
    codes[129, 3], codes[129, 4] = 5, 9
    byte[129, 16], byte[37, 6] = 77, 33
    c, s = O.pack(codes, byte, "nvfp4")
    # row 129: row 1 of the second row tile, whose first k-tile is number 2; its
    # unit 0 (columns 0 - 31) is the second 16 bytes
    assert c.size == 4 * 16384
    at = 2 * 16384 + 128 + 16
    assert c[at + 1] == 0x50 and c[at + 2] == 0x09
    assert np.count_nonzero(c) == 2
    assert s.size == 2 * 2 * 2048
    # row 129: second row tile, row 1 of it; block 16: second k-tile, block 0
    assert s[(1 * 2 + 1) * 2048 + 16] == 77
    # row 37: row 5 of the second group of 32; block 6: second word, third byte
    assert s[512 + 5 * 16 + 1 * 4 + 2] == 33


def test_the_block_is_the_plain_one_where_quantisation_loses_nothing():
    r = rng(6)
    X = r.choice([0.0, 1, 2, -4, 6], (4, 32))
    X[:, 0] = 6
    A = r.choice([0.0, 1, -2, 6], (32, 16))
    A[0] = 6
    B = r.choice([0.0, 0.5, -1], (16, 32))
    got = O.mlp_forward(X, A, B, "mxfp4", gelu=lambda h: np.sign(h) * 4)
    assert np.array_equal(got["H"], X @ A)
    assert np.array_equal(got["Z"], (np.sign(X @ A) * 4) @ B)
    f = O.mlp_forward(X, A, B, "nvfp4")
    assert np.allclose(f["Y"], OM.gelu(f["H"]), rtol=0, atol=1e-12)
