"""How far a value in the 8-bit cache may be from what was written, by its definition."""
import numpy as np
import pytest

import more_serve_ref as more


def rounded(x, exponents):
    """What is left of x [16, 1, 64] after a write with exponents[0], and after raises to the others."""
    codes = more.e4m3(x * 2.0 ** -exponents[0])
    for old, new in zip(exponents, exponents[1:]):
        codes = more.e4m3(more.values(codes) * 2.0 ** (old - new))
    return more.values(codes) * 2.0 ** exponents[-1]


def bound(x, e):
    return 2.0 ** -4 * np.abs(x) + 2.0 ** -9 * 2.0 ** e


def test_a_value_that_is_rounded_as_a_normal_and_as_a_subnormal_code():
    x = np.array([11.51 * 2.0 ** -12])
    got = rounded(x, [-3, 0])
    assert got == 2.0 ** -8 and np.abs(got - x) > 2.0 ** -4 * x and np.abs(got - x) > 2.0 ** -10  # neither alone
    assert (np.abs(got - x) <= bound(x, 0)).all()


@pytest.mark.parametrize("raises", [0, 1, 2, 5, 12])
def test_values_after_any_number_of_raises(raises):
    rng = np.random.default_rng(raises)
    for _ in range(200):
        e = np.concatenate([[rng.integers(-32, 10)], rng.integers(1, 4, raises)]).cumsum().clip(max=32)
        x = rng.uniform(-448, 448, 300) * 2.0 ** (e[0] - rng.integers(0, 20, 300))
        assert (np.abs(rounded(x, e.tolist()) - x) <= bound(x, e[-1])).all()


@pytest.mark.parametrize("d", [64, 128])
def test_tokens_that_come_one_by_one(d):
    """The same through the cache's blocks: each token may raise the exponent."""
    rng = np.random.default_rng(d)
    for _ in range(5):
        pages = np.zeros((1, 32 * d + 16), np.uint8)
        x = rng.standard_normal((2, 16, 1, d)) * 2.0 ** rng.integers(-40, 30, (2, 16, 1, 1))
        for t in range(16):
            more.append8(pages, 16, 1, d, x[0, t:t + 1], x[1, t:t + 1], [t])
        got = more.read8(pages, 16, 1, d, range(16))
        for n in range(2):
            e = int(pages[0, 32 * d + n:32 * d + n + 1].view(np.int8)[0])
            assert (np.abs(got[n] - x[n]) <= bound(x[n], e)).all()
