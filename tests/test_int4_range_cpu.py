"""The largest rows of the cache in 4 bits: a row of finite range stands for finite values."""

import numpy as np

from oracle import int4

LARGEST = np.finfo(np.float32).max


def rows_at_the_top(count=2000):
    """fp32 rows whose range goes up to the largest float, and not beyond."""
    rng = np.random.default_rng(0)
    x = rng.uniform(0, 1, (count, 64))
    low = rng.uniform(0, 1, count)
    low[:4] = 0, 1, 0.5, 1e-3
    span = LARGEST * np.where(np.arange(count) < 8, 1.0, rng.uniform(0.9, 1, count))
    y = (x - low[:, None]) * (span / 2)[:, None]
    y[:, 0], y[:, 1] = -low * span, (1 - low) * span * (1 - 2.0**-23)
    return y.astype(np.float32)


def test_rows_of_finite_range_stand_for_finite_values():
    x = rows_at_the_top()
    with np.errstate(over="ignore"):
        fine = np.isfinite(x.max(-1) - x.min(-1))
    assert fine.sum() > 1900
    n, s, z = int4.quantise(x[fine])
    assert s.max() == 1.125 * 2.0**124
    y = int4.stands_for(n, s, z)
    assert (np.abs(y) <= LARGEST).all()
    assert (np.abs(n - z[:, None])[s == s.max()] <= 14).all()
    assert np.isnan(int4.round_trip(x[~fine])).all()


def test_the_bound_by_arithmetic():
    # at the largest step |x| / s is below 2^128 / (1.125 * 2^124) = 14.3, which rounds to 14;
    # at the next one 15 steps are 15 * 2^124
    for s, most in ((1.125 * 2.0**124, 14), (2.0**124, 15)):
        assert most * s <= LARGEST
    assert 2.0**128 / (1.125 * 2.0**124) < 14.5
    # a range of the largest float is rounded up to the largest step, no further
    assert 2.0**124 < float(LARGEST) / 15 < 1.125 * 2.0**124
