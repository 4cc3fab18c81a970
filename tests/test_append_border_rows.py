"""The inputs of the border test, on the CPU: their largest values do lie next to the border, on both
sides of it, and an fp32 evaluation picks the wrong exponent for some of them."""

import numpy as np

import oracle
from tests._borders import BORDER, border_rows, exponents, rows_in


def test_border_rows_are_decided_by_fp64_alone():
    theta, first = oracle.rope_theta(64, 10000.0), 100_000
    x, gamma = border_rows(400, first, theta, 1)
    rows = rows_in(np.float64, x, gamma, first, theta)
    most = np.abs(rows).max(axis=1)
    assert np.all(np.abs(most / BORDER - 1) < 2.0 ** -21)
    latent = np.abs(rows[:, :512]).max(axis=1) == most
    assert np.array_equal(latent, np.arange(400) % 2 == 0)
    want, got = exponents(rows), exponents(rows_in(np.float32, x, gamma, first, theta))
    for kind in (0, 1):     # latent and rotated values
        assert set(want[kind::2]) == {-7, -6}
        assert (want[kind::2] != got[kind::2]).sum() >= 10
