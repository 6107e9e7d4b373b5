"""Pins of the oracle of caches held in 4 bits: the form's promises, over every scale and
magnitude, and the margins that let binary32 decide as exact arithmetic does."""
import numpy as np
import pytest

from oracle import paged_cache as pc
from oracle import quant_cache as qc


def halves():
    return np.arange(0x7C00, dtype=np.uint16).view(np.float16)


def test_scales_have_8_bits_and_numbers_are_exact():
    assert (np.diff(qc.SCALES) > 0).all() and qc.SCALES[1] == 2.0 ** -24 and qc.SCALES[-1] == 9344
    for n in range(8):
        x = n * qc.SCALES
        assert (x.astype(np.float16).astype(np.float64) == x).all()


def test_every_magnitude_has_the_smallest_scale_that_reaches_it():
    a = halves().astype(np.float64)
    x = np.zeros((len(a), 32), np.float16)
    x[:, 5] = halves()
    x[::2, 5] *= -1
    n, s = qc.quantise(x, 32)
    s = s[:, 0, 0]
    reached = a <= 7 * 9344
    assert (7 * s[reached] >= a[reached]).all()
    below = qc.SCALES[np.maximum(np.searchsorted(qc.SCALES, s) - 1, 0)]
    assert ((7 * below < a) | (s == 0)).all()
    assert (n >= 1).all() and (n <= 15).all()
    assert (np.abs((n[:, 0, 0, 5] - 8.0) * s - x[:, 5]) <= s / 2).all()
    # in binary32, with a margin: what the kernel computes
    q = (halves().astype(np.float32) * np.float32((1 - 2.0 ** -20) / 7))
    up = ((q.view(np.uint32) + 0xFFFF) & 0xFFFF0000).view(np.float32)
    low = np.ceil(q * np.float32(2.0 ** 24)) * np.float32(2.0 ** -24)
    assert (np.minimum(np.where(q < 2.0 ** -16, low, up), 9344) == s).all()


def test_codes_in_binary32_are_the_exact_ones():
    """Every pair of a scale's 8 and a number's 11 bits, at every distance of their exponents
    that gives a code; ties go up."""
    S = np.arange(128, 256)[:, None]
    X = np.arange(1024, 2048)[None, :]
    for e in range(-14, 3):
        x = X * 2.0 ** e
        q = x / S
        keep = (q < 7.02) & (q > 0.01)
        for sign in (1, -1):
            exact = np.floor(sign * q + 0.5)[keep]  # a quotient of small whole numbers that is a half is exact
            inv = (np.float32(1) / S.astype(np.float32)) * np.ones_like(q, np.float32)
            for slack in (-1, 0, 1):  # a reciprocal that is off by its last bit
                r = np.nextafter(inv, np.float32(np.inf) * slack) if slack else inv
                f = (sign * x * r.astype(np.float64) + (8.5 + 2.0 ** -14)).astype(np.float32)
                assert (np.floor(f[keep]) - 8 == exact).all()
    tie = np.zeros((1, 32), np.float16)
    tie[0, :4] = 7, 2.5, -2.5, -0.5
    n, s = qc.quantise(tie, 32)
    assert s == 1 and (n[0, 0, 0, :4] == [15, 11, 6, 8]).all()


@pytest.mark.parametrize("C,d", [(128, 64), (400, 80), (24, 8), (96, 96), (512, 256), (36 * 8, 72)])
def test_rows_hold_what_they_stand_for(C, d):
    rng = np.random.default_rng(C + d)
    x = (rng.standard_normal((50, C)) * np.exp(rng.uniform(-12, 9, (50, 1)))).astype(np.float16)
    x[3] = 0
    x[4, 1], x[5, C - 1], x[6, d // 2] = np.nan, np.inf, -np.inf
    row = qc.sizes(C, d)[3]
    before = rng.integers(0, 256, (50, row), dtype=np.uint8)
    rows = qc.rows_of(x, d, before)
    used = qc.sizes(C, d)[2] + 2 * (C // d) * qc.sizes(C, d)[1]
    assert row % 16 == 0 and row - used < 16 and (rows[:, used:] == before[:, used:]).all()
    y = qc.numbers(rows, C, d).astype(np.float64)
    n, s = qc.quantise(x, d)
    per = np.repeat(s, 32, -1).reshape(50, C // d, -1)[:, :, :d].reshape(50, C)
    ok = np.isfinite(per)
    assert (np.isnan(y) == ~ok).all() and (np.abs(y - x.astype(np.float64))[ok] <= per[ok] / 2).all()
    for t, c in ((4, 1), (5, C - 1), (6, d // 2)):
        g = c % d // 32
        assert np.isnan(y[t].reshape(-1, d)[c // d, 32 * g:32 * g + 32]).all()
    # held numbers are held again as they are
    again = qc.numbers(qc.rows_of(y.astype(np.float16), d, before), C, d)
    assert np.array_equal(again.astype(np.float64)[ok], y[ok])


def test_slots():
    c = pc.empty(1, 10, 4, 16, 3, 6)
    st, got = pc.reserve(c, [0, 2], [0, 6, 9], 9)
    assert st == 0
    st, s = qc.slots(c, [0, 2, 0], None, [0, 6, 9, 11], 12)
    assert st == 0 and (s[:9] == got).all() and (s[9:11] == got[:2]).all() and s[11] == -1
    st, s = qc.slots(c, [0, 2, 1], [3, 2, 0], [1, 4, 5, 5], 6)
    assert st == 0 and s.tolist() == [-1, *got[3:6], got[8], -1]
    for bad in ([[0], [1], [0, 6]], [[3], None, [0, 1]], [[-1], None, [0, 1]], [[1], None, [0, 1]], [[0], [-1], [0, 1]],
                [[0], None, [0, 7]], [[0], None, [4, 2]]):
        st, s = qc.slots(c, *bad, 6)
        assert st == pc.REFUSED and (s == -1).all()
