"""The packed activations' split, without a GPU: numpy's IEEE halves on the
stated arithmetic.  x' = x 2^(15 - E) with max |x| in [2^(E-1), 2^E); f32 rows
as hi = f16(x') and lo = f16(x' - hi), bf16 rows as f16(x').  The bounds are
those that include/qgemv.h states, worst where the maximum is a power of two."""
import numpy as np
import pytest


def scaled(x, peak):
    return np.ldexp(x.astype(np.float64), 15 - np.frexp(peak)[1]).astype(np.float32)


def f32_error(x, peak):
    """|hi + lo - x'| in units of x."""
    t = scaled(x, peak)
    hi = t.astype(np.float16)
    lo = (t - hi.astype(np.float32)).astype(np.float16)
    back = hi.astype(np.float64) + lo.astype(np.float64)
    return np.abs(np.ldexp(back, np.frexp(peak)[1] - 15) - x.astype(np.float64))


def bf16_values(n, lo, hi, rng):
    m = (rng.integers(128, 256, n) / 128.0) * 2.0 ** rng.integers(lo, hi, n)
    return m.astype(np.float32)


@pytest.mark.parametrize("peak", [1.0, 1.9999, 2.0 ** 90, 3.0e-30])
def test_f32_split(peak):
    rng = np.random.default_rng(0)
    e = rng.uniform(-60.0, 0.0, 400000)
    x = (peak * 2.0 ** e * rng.choice([-1, 1], e.size)).astype(np.float32)
    err = f32_error(x, np.float32(peak))
    mag = np.abs(x.astype(np.float64))
    big = mag >= 2.0 ** -17 * peak
    assert np.all(err[big] <= 2.0 ** -22 * mag[big])
    assert np.all(err[~big] <= 2.0 ** -39 * peak)
    if peak == 1.0:              # and no tighter ones hold
        assert (err[~big].max() > 2.0 ** -40 * peak)
        some = (mag >= 2.0 ** -18 * peak) & ~big
        assert np.any(err[some] > 2.0 ** -22 * mag[some])


@pytest.mark.parametrize("peak", [1.0, 1.9921875, 2.0 ** 90])
def test_bf16_split(peak):
    rng = np.random.default_rng(1)
    x = bf16_values(400000, -60, 0, rng) * np.float32(peak if peak > 2 else 1.0) / 2
    t = scaled(x, np.float32(peak))
    err = np.abs(np.ldexp(t.astype(np.float16).astype(np.float64), np.frexp(peak)[1] - 15) -
                 x.astype(np.float64))
    mag = np.abs(x.astype(np.float64))
    big = mag >= 2.0 ** -28 * peak
    assert np.all(err[big] == 0.0)
    assert np.all(err[~big] <= 2.0 ** -39 * peak)
