"""The oracle of the int8 codes and their products against closed forms."""
import numpy as np
import pytest

import oracle as O


@pytest.mark.parametrize("a", [1.0, 127.0, 3e38, 2.0 ** -99, 1e-3])
def test_scales_and_codes_closed_forms(a):
    x = np.float32(a) * np.array([[1.0, -1.0, 0.0, 0.5]], np.float32)
    c, s = O.int8.quantize(x)
    assert s[0] == np.float32(np.float64(x[0, 0]) / 127) and s.dtype == np.float32
    # 63.5 goes to the even neighbour, or past it where the product of two roundings does
    assert c[0, :3].tolist() == [127, -127, 0] and c[0, 3] in (63, 64)
    np.testing.assert_array_equal(O.int8.quantize(np.float32([[127.0, 63.5, 62.5, -0.5]]))[0], [[127, 64, 62, 0]])


def test_rows_without_a_grid_and_tiny_rows():
    x = np.zeros((5, 6), np.float32)
    x[1, 3], x[2, 0], x[3] = np.nan, -np.inf, 1e-42
    x[4] = 2.0 ** -101
    c, s = O.int8.quantize(x)
    assert np.isnan(s[1]) and np.isnan(s[2]) and not c[:4].any()
    assert s[0] == s[3] == s[4] == np.float32(2.0 ** -100 / 127) and (c[4] == 64).all()


def test_codes_are_the_nearest_multiples():
    x = np.random.default_rng(0).standard_normal((40, 500)).astype(np.float32)
    c, s = O.int8.quantize(x)
    assert c.min() >= -127 and np.abs(c).max(1).tolist() == [127] * 40
    q = x.astype(np.float64) / s[:, None].astype(np.float64)
    assert np.all(np.abs(q - c) <= 0.5 + 2.0 ** -14)          # four roundings of up to 127


def test_products_of_whole_numbers():
    r = np.random.default_rng(1)
    x, w = r.integers(-128, 128, (4, 300)), r.integers(-128, 128, (3, 5, 300))
    one = np.ones(5)
    y, mag = O.int8.matmul(x, np.ones(4), w[0], one, np.arange(5.0))
    np.testing.assert_array_equal(y, x @ w[0].T + np.arange(5))
    assert np.all(mag >= np.abs(y))
    y, _, has = O.int8.grouped(x, np.ones(4), w, np.ones((3, 5)), [1, 3, 3, 5], [0, 2, 2, 3, 4, 1])
    np.testing.assert_array_equal(y[1:3], x[[2, 2]] @ w[0].T)
    np.testing.assert_array_equal(y[3], x[3] @ w[2].T)
    assert np.isnan(y[4]).all() and has.tolist() == [False, True, True, True, True, False]
