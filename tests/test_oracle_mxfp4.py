"""Pins of the MXFP4 oracle: exponents and codes against exact rational arithmetic, products against plain loops."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import mxfp4
from oracle.codec import bf16_to_f32, f32_to_bf16

MAGS = [Fraction(0), Fraction(1, 2), Fraction(1), Fraction(3, 2), Fraction(2), Fraction(3), Fraction(4), Fraction(6)]


def _value(bits):
    return Fraction(float(bf16_to_f32(np.array([bits], np.uint16))[0]))


def _exponent(amax, rule):
    """By searching: the smallest X with amax <= 6 2^X, or the largest with 2^(X + 2) <= amax."""
    if amax == 0:
        return -127
    x = 200
    if rule == "ceil":
        while amax <= 6 * Fraction(2) ** (x - 1):
            x -= 1
    else:
        while Fraction(2) ** (x + 2) > amax:
            x -= 1
    return min(max(x, -127), 127)


def _nearest(v, negative):
    """By distance to every magnitude; a tie to the even code; saturating."""
    a = abs(v)
    best = min(range(8), key=lambda c: (abs(a - MAGS[c]), c % 2))
    return best | (8 if negative else 0)


@pytest.mark.parametrize("rule", ["ceil", "floor"])
def test_codes_and_scales_against_rationals(rule):
    rng = np.random.default_rng(3)
    blocks = [rng.integers(0, 0x7F80, 32).astype(np.uint16) for _ in range(20)]                # any magnitudes
    for top in (0x40C0, 0x40C1, 0x40BF, 0x4100, 0x0001, 0x0080, 0x0100, 0x01C0, 0x7F7F, 0x7F40, 0x0000):
        b = (top - np.minimum(rng.integers(0, 0x300, 32), top)).astype(np.uint16)
        b[5] = top
        blocks.append(b)
    tie = f32_to_bf16(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4, np.float32))
    blocks.append(tie)
    x = np.stack(blocks).astype(np.uint16) | (rng.integers(0, 2, (len(blocks), 32)).astype(np.uint16) << 15)
    q, s, dq = mxfp4.quantize(x, rule)
    for i, row in enumerate(x):
        vals = [_value(b) for b in row]
        e = _exponent(max(abs(v) for v in vals), rule)
        assert s[i, 0] == e + 127, (i, s[i, 0], e)
        for j, v in enumerate(vals):
            code = int(q[i, j // 2] >> (4 * (j & 1))) & 15
            want = _nearest(v / Fraction(2) ** e, row[j] >> 15)
            assert code == want, (i, j, code, want)
            back = (-1 if code & 8 else 1) * MAGS[code & 7] * Fraction(2) ** e
            got = bf16_to_f32(dq[i, j:j + 1])[0]
            assert np.isinf(got) if abs(back) >= Fraction(2) ** 128 else Fraction(float(got)) == back


def test_matrix_and_products_against_loops():
    rng = np.random.default_rng(4)
    q, s = rng.integers(0, 256, (5, 32)).astype(np.uint8), rng.integers(120, 134, (5, 2)).astype(np.uint8)
    w = mxfp4.matrix(q, s)
    for i in range(5):
        for j in range(64):
            code = int(q[i, j // 2] >> (4 * (j & 1))) & 15
            assert w[i, j] == (-1 if code & 8 else 1) * float(MAGS[code & 7]) * 2.0 ** (int(s[i, j // 32]) - 127)
    s[2, 1] = 255
    assert np.isnan(mxfp4.matrix(q, s)[2, 32:]).all() and np.isfinite(mxfp4.matrix(q, s)[2, :32]).all()
    a8 = np.arange(256, dtype=np.uint8).reshape(8, 32) & 0x77
    assert mxfp4.matrix8(a8, np.full((8, 1), 128, np.uint8))[1, 0] == 2.0 * mxfp4.matrix8(a8, np.full((8, 1), 127, np.uint8))[1, 0]
    x, wg = rng.standard_normal((6, 4)), rng.standard_normal((3, 2, 4))
    off, row = [0, 2, 2, 5], np.array([5, 0, 3, 3, 9, 1])
    y = mxfp4.grouped(x, wg, off, row, keep=np.full((6, 2), 7.0))
    dy = rng.standard_normal((6, 2))
    dx, dw = mxfp4.dgrad(dy, wg, off), mxfp4.wgrad(dy, x, off, row)
    want = np.zeros_like(dw)
    for i, g in enumerate([0, 0, 2, 2, 2]):
        at = min(row[i], 5)
        assert np.allclose(y[i], [sum(x[at, c] * wg[g, n, c] for c in range(4)) for n in range(2)])
        assert np.allclose(dx[i], sum(dy[i, n] * wg[g, n] for n in range(2)))
        want[g] += np.outer(dy[i], x[at])
    assert np.all(y[5] == 7.0) and np.all(dx[5] == 0) and np.allclose(dw, want) and np.all(dw[1] == 0)


def test_gradients_against_differences():
    """The gradients of sum(dy * y) by central differences (y is linear in x and in w, so they are exact)."""
    rng = np.random.default_rng(5)
    x, w, off = rng.standard_normal((5, 3)), rng.standard_normal((2, 4, 3)), [0, 2, 5]
    row = np.array([4, 1, 0, 4, 2])
    dy = rng.standard_normal((5, 4))

    def loss(x, w):
        return float((dy * mxfp4.grouped(x, w, off, row)).sum())

    dx, dw = mxfp4.dgrad(dy, w, off), mxfp4.wgrad(dy, x, off, row)
    for i in range(5):
        for j in range(3):
            d = np.zeros_like(x)
            d[i, j] = 0.5
            of_row = sum(dx[t, j] for t in range(5) if row[t] == i)     # a row read twice collects both
            assert abs(loss(x + d, w) - loss(x - d, w) - of_row) < 1e-12
    for g in range(2):
        for i in range(4):
            for j in range(3):
                d = np.zeros_like(w)
                d[g, i, j] = 0.5
                assert abs(loss(x, w + d) - loss(x, w - d) - dw[g, i, j]) < 1e-12
