"""The float64 references of the 16-bit expert FFN and of INT8, pinned: the
gradients against central differences of the forward form, the forward forms
against a loop over single elements, the quantiser against exact rationals."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import experts16 as X
from oracle import int8 as Q

OFF = np.array([0, 3, 3, 7])


def _inputs(seed=0, I=4, H=6):
    r = np.random.default_rng(seed)
    rows = r.integers(0, 5, 7)
    return r.standard_normal((5, H)), r.standard_normal((3, 2 * I, H)) * 0.5, r.standard_normal((7, I)), rows


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_gradients_against_differences(kind):
    x, w, dh, rows = _inputs()

    def loss(x_, w_):
        return float((X.gated(x_, w_, OFF, rows, kind)[0][0] * dh).sum())

    (dx, _), (dw, _) = X.gated_grad(dh, x, w, OFF, rows, kind)
    eps = 1e-5                     # central differences: error eps^2 f''' / 6 + 2^-53 |f| / eps, far below 1e-6
    dtok = np.zeros_like(x)
    np.add.at(dtok, rows, dx)      # the gradient of a gathered row is the sum over its copies
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = eps
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * eps) - dtok[i]) < 1e-6
    for i in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[i] = eps
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * eps) - dw[i]) < 1e-6
    assert not dw[1].any()         # the expert without rows


def test_product_gradients_against_differences():
    x, w, _, rows = _inputs(1)
    dy = np.random.default_rng(2).standard_normal((7, w.shape[1]))
    (da, _), (db, _) = X.product_grad(dy, x, w, OFF, rows)
    y = X.product(x, w, OFF, rows)[0]
    for p in range(7):
        e = 0 if p < 3 else 2
        assert np.allclose(y[p], [sum(x[rows[p], k] * w[e, n, k] for k in range(6)) for n in range(8)], rtol=1e-13)
        assert np.allclose(da[p], [sum(dy[p, n] * w[e, n, k] for n in range(8)) for k in range(6)], rtol=1e-13)
    eps = 1e-5
    for i in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[i] = eps
        diff = ((X.product(x, w + d, OFF, rows)[0] - X.product(x, w - d, OFF, rows)[0]) * dy).sum() / (2 * eps)
        assert abs(diff - db[i]) < 1e-6


def test_int8_quantizer_against_rationals():
    r = np.random.default_rng(3)
    x = np.concatenate([r.standard_normal((6, 16)) * 10.0 ** r.integers(-20, 20, (6, 1)), np.zeros((1, 16))])
    x = x.astype(np.float32)
    codes, s = Q.quantize(x)
    assert s[-1] == 1 and not codes[-1].any()
    for i in range(6):
        # two roundings, of 1/127 and of the product: (1 + 2^-24)^2 - 1 < 2^-22.99
        assert abs(Fraction(float(s[i])) * 127 / Fraction(float(np.abs(x[i]).max())) - 1) <= Fraction(101, 100 * 2 ** 23)
        assert np.abs(codes[i]).max() == 127
        for j in range(16):
            # within half a step of the rational quotient, and a float32 rounding of it
            q = Fraction(float(x[i, j])) / Fraction(float(s[i]))
            assert abs(int(codes[i, j]) - q) <= Fraction(1, 2) + abs(q) / 2 ** 24
    tie = np.zeros((1, 8), np.float32)
    tie[0, :4] = [127, 2.5, -3.5, 0.5]             # scale 1 (the product rounds to it): ties go to the even code
    codes, s = Q.quantize(tie)
    assert s[0] == 1 and codes[0, :4].tolist() == [127, 2, -4, 0]


def test_int8_product_brute_force():
    r = np.random.default_rng(4)
    a, b = r.integers(-128, 128, (5, 16)).astype(np.int8), r.integers(-128, 128, (3, 4, 16)).astype(np.int8)
    sa, sb = r.random(5).astype(np.float32), r.random((3, 4)).astype(np.float32)
    rows = r.integers(0, 5, 7)
    y, tol = Q.grouped_gemm(a, sa, b, sb, OFF, rows)
    for p in range(7):
        e = 0 if p < 3 else 2
        for n in range(4):
            want = sum(int(a[rows[p], k]) * int(b[e, n, k]) for k in range(16)) * float(sa[rows[p]]) * float(sb[e, n])
            assert abs(y[p, n] - want) <= 1e-12 * abs(want)
    assert (tol >= 0).all()
