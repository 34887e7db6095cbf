"""The 8-bit states' dither, as the oracle defines it: each number goes to one of
its two neighbours on E4M3's grid with the mean kept, and the states follow
binary32 ones where rounding to nearest stops.

Tolerances.  A mean over n evenly spread places in a step has a standard
deviation of at most half a step / sqrt(n); five of them are allowed.  For states
over many steps see states_tolerance."""

import numpy as np
import pytest

from oracle import adamw as A
from oracle import formats as F

GRID = np.sort(np.unique(np.abs(F.decode(np.arange(127, dtype=np.uint8), "e4m3"))))


def states_tolerance(numbers):
    """Of the mean of sqrt(v8) / sqrt(v32), and of its root mean square error.

    One rounding of a root q between two numbers of the grid h apart (h <= q / 8)
    has variance f (1 - f) h^2 <= |d| h, d the way to the nearer one.  The root
    was on the grid a step before, so d is its move and the scale's, each at most
    (1 - b2) / 2 |g^2 / v - 1| of it, on average below (1 - b2) / 2: variance (1 -
    b2) / 8 of q^2 a step.  The moves shrink a deviation by (1 - b2) / 2 of itself
    a step, so its variance settles at (1 - b2) / 8 / (1 - b2) = 1 / 8, 0.36 of the
    root.  The mean of `numbers` roots is then off by 0.36 / sqrt(numbers), five of
    which are allowed, and by a second-order term of 1 / 64."""
    sd = 8 ** -0.5
    return 5 * sd / numbers ** 0.5 + 1 / 64, sd


@pytest.mark.parametrize("q", [448.0, 447.99, 3.7, 1.0, 1.0625, 0.0156251, 2.0 ** -6, 0.0151, 2.0 ** -9, 1.3e-3, 3e-6, 0.0])
def test_one_of_the_two_neighbours_with_the_mean_kept(q):
    q = np.float32(q)
    r = (np.arange(4096, dtype=np.uint32) * 256 + 17)  # evenly over [0, 2^20)
    y = A.dithered(np.full(r.size, q), r)
    low = GRID[GRID <= q].max()
    high = GRID[GRID >= q].min()
    assert set(np.unique(y)) <= {low, high}
    assert abs(y.mean(dtype=np.float64) - q) <= (high - low) / r.size + q * 2.0 ** -24 + 2.0 ** -30
    np.testing.assert_array_equal(A.dithered(np.full(r.size, -q), r), -y)


def test_the_dither_is_spread_over_numbers_and_steps():
    """Means of the 20 bits over 2048 numbers (of one step) and over 2048 steps (of
    one number): five standard deviations, 0.29 / sqrt(2048) each.  Correlations of
    one number's steps, and of numbers a multiple of four apart (four share a
    word): six, of at least 2048^2 / 2 and 2048^2 / 8 / 8 pairs."""
    n = 2048
    h = np.stack([A.dither(n, t) for t in range(1, n + 1)])
    for bits in (h >> np.uint32(12), h & np.uint32(0xFFFFF)):
        u = bits / 2.0 ** 20
        assert np.abs(u.mean(0) - 0.5).max() <= 5 * 12 ** -0.5 / n ** 0.5
        assert np.abs(u.mean(1) - 0.5).max() <= 5 * 12 ** -0.5 / n ** 0.5
        for d in (1, 2, 3, 4, 64, 500):  # correlations over 2048^2 and a quarter of it
            assert abs(np.corrcoef(u[:-d].ravel(), u[d:].ravel())[0, 1]) <= 6 / n
            assert abs(np.corrcoef(u[:, :-4 * d:4].ravel(), u[:, 4 * d::4].ravel())[0, 1]) <= 6 * 2 * 8 ** 0.5 / n


def follow(betas, dither, steps, numbers=1024, seed=3):
    """Ratios of the 8-bit roots to the binary32 ones; from step 300 on every
    second number's gradients are a twentieth."""
    rng = np.random.default_rng(seed)
    low = np.arange(numbers) % 2 == 0
    zero = np.zeros(numbers, np.float32)
    m, v, m8, v8 = (zero.copy() for _ in range(4))
    kw = dict(lr=0.0, betas=betas, eps=1e-8, weight_decay=0.0)
    for t in range(1, steps + 1):
        g = (rng.normal(size=numbers) * 1e-3 * np.where(low & (t > 300), 0.05, 1.0)).astype(np.float32)
        _, m, v = A.step32(zero, g, m, v, t, **kw)
        _, m8, v8 = A.step32(zero, g, m8, v8, t, **kw)
        root = np.sqrt(v8)
        s, q = A.scales(m8), A.scales(root)
        m8 = A.values(A.codes(m8, s, step=t if dither else None), s)
        root = A.values(A.codes(root, q, True, step=t if dither else None), q)
        v8 = root * root
    return np.sqrt(v8 / v)[low], np.sqrt(v8 / v)[~low]


@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.9, 0.99), (0.9, 0.97), (0.97, 0.95)])
def test_dithered_states_follow(betas):
    assert A.dithers(betas)
    mean, sd = states_tolerance(512)
    for r in follow(betas, True, 700):
        assert abs(r.mean() - 1) <= mean and np.sqrt(np.mean((r - 1) ** 2)) <= sd + mean


def test_states_to_nearest_follow_up_to_the_rules_limit_and_not_beyond():
    """A root that nearest holds is off by half a step, 2^-4 of it at most, and by
    what the gradients' noise has not moved it by yet, as much again."""
    assert not A.dithers((0.9, 0.95)) and not A.dithers((0.94, 0.95))
    for r in follow((0.9, 0.95), False, 700):
        assert abs(r.mean() - 1) <= 2 * 2.0 ** -4
    fallen, _ = follow((0.9, 0.999), False, 700)
    assert fallen.mean() > 1.5
