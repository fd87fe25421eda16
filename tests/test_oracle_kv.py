"""Pins of the oracle's rotary positions and attention by properties that do not re-use their
formulas: complex rotation, relative positions, hand-worked masks and weights."""

import numpy as np
import pytest

from oracle import attention as oat


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_complex_rotation(interleaved):
    g = np.random.default_rng(1)
    x, pos = g.standard_normal((5, 3, 12)), np.array([0, 1, 7, -3, 1000])
    f = np.array([1.0, 0.3, 0.01, 1e-4])
    y = oat.rope(x, pos, f, 8, interleaved, gain=1.5)
    a = slice(0, 8, 2) if interleaved else slice(0, 4)
    b = slice(1, 8, 2) if interleaved else slice(4, 8)
    z = (x[..., a] + 1j * x[..., b]) * 1.5 * np.exp(1j * pos[:, None, None] * f)
    np.testing.assert_allclose(y[..., a], z.real, atol=1e-12)
    np.testing.assert_allclose(y[..., b], z.imag, atol=1e-12)
    np.testing.assert_array_equal(y[..., 8:], x[..., 8:])


def test_rope_products_depend_on_the_distance_alone():
    g = np.random.default_rng(2)
    q, k = g.standard_normal((1, 1, 16)), g.standard_normal((1, 1, 16))
    f = 10000.0 ** (-np.arange(0, 16, 2) / 16)
    dots = [np.sum(oat.rope(q, [p + 5], f, 16) * oat.rope(k, [p], f, 16)) for p in (0, 3, 100000)]
    np.testing.assert_allclose(dots, dots[0], atol=1e-10)


def test_rope_transposed_is_the_gradient():
    g = np.random.default_rng(3)
    x, w = g.standard_normal((4, 2, 10)), g.standard_normal((4, 2, 10))
    f, pos = np.array([0.7, 0.02, 0.5]), np.array([3, 9, 81, 6561])
    for il in (False, True):
        y = oat.rope(x, pos, f, 6, il, gain=1.3)
        grad = oat.rope(w, pos, f, 6, il, gain=1.3, transposed=True)
        np.testing.assert_allclose(np.sum(y * w), np.sum(x * grad), rtol=1e-12)
        # differences: the map is linear, so a difference of step 1 is exact up to rounding
        d = np.zeros_like(x)
        d[2, 1, 4] = 1.0
        diff = np.sum((oat.rope(x + d, pos, f, 6, il, gain=1.3) - y) * w)
        np.testing.assert_allclose(diff, grad[2, 1, 4], rtol=1e-9)


def test_seen_by_hand():
    assert oat.seen(5, 2, 0).tolist() == [True, True, True, True, False]
    assert oat.seen(5, 2, 1).tolist() == [True] * 5
    # three drafted tokens after two: the third sees the first and itself, not the second
    assert oat.seen(5, 3, 2, [1, 0, 1]).tolist() == [True, True, True, False, True]
    assert oat.seen(2, 3, 0).tolist() == [False, False]      # a query before the first token
    assert oat.seen(2, 2, 0, [0, 0]).tolist() == [False, False]


def test_attend_by_hand():
    k = np.array([[1.0, 0.0], [0.0, 1.0], [5.0, 5.0]])
    v = np.array([[1.0, 0.0], [0.0, 1.0], [100.0, 100.0]])
    out, p = oat.attend(np.array([np.log(3.0), 0.0]), k, v, 1.0, np.array([True, True, False]))
    np.testing.assert_allclose(p, [0.75, 0.25, 0.0])
    np.testing.assert_allclose(out, [0.75, 0.25])
    out, p = oat.attend(np.array([1.0, 1.0]), k, v, 1.0, np.zeros(3, dtype=bool))
    assert not out.any() and not p.any()
