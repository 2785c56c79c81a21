"""Pins of the 8-bit cache's plain forms: codes, rounding, exponents."""
import numpy as np
import pytest

from tests import kv8_ref as r


def test_codes_are_those_of_the_type():
    torch = pytest.importorskip("torch")
    got = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(got, r.CODES, equal_nan=True)


def test_rounding_is_to_nearest_even():
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(1).normal(size=5000) * 2.0 ** np.random.default_rng(2).integers(-12, 8, 5000)
    x = np.concatenate([x, np.array([2.0 ** -10, 3 * 2.0 ** -10, 17.0, 18.0, 19.0, 448.0, -448.0, 0.0, 1.0625, 1.1875])])
    x = x[np.abs(x) <= 448].astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(r.rounded(x.astype(np.float64), 127), want)


def test_exponents():
    top = np.array([448.0, 448.0001, 1.75, 1.7500001, 0.0, 2.0 ** -80, 1.0, 3.0e38])
    e = r.exponent(top)
    assert e.tolist() == [127, 128, 119, 120, 63, 63, 119, 127 + 120]
    assert (top <= 448 * 2.0 ** (e - 127.0)).all()
    assert (top[[1, 3, 6, 7]] > 448 * 2.0 ** (e[[1, 3, 6, 7]] - 128.0)).all()


def test_rotation_keeps_lengths_and_adds_angles():
    x = np.random.default_rng(3).normal(size=(5, 2, 64))
    f = 10000.0 ** (-np.arange(16) / 16)
    for inter in (False, True):
        y = r.rotate(x, np.arange(5) * 7, f, inter)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[..., 32:], x[..., 32:])
        assert np.allclose(r.rotate(y, np.arange(5), f, inter), r.rotate(x, np.arange(5) * 8, f, inter))
        assert np.array_equal(y[0], x[0])
