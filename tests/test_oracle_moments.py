"""The oracle of 8-bit moments with stochastic rounding: its bits, its codes by
hand, and that moments rounded so follow their gradients over many steps."""

import numpy as np
import pytest

from oracle import moments as M


def group(*first):
    v = np.zeros(32)
    v[:len(first)] = first
    return v


def test_random_bits():
    """2^22 of them: means, neighbours in place and in step, and a bit's effect, each to 5 standard deviations."""
    n, steps = 1 << 16, 64
    h = np.stack([M.dice(5, t, np.arange(n)) for t in range(1, steps + 1)])
    sd = 1 / np.sqrt(h.size)
    for u in M.fractions(h):
        assert abs(u.mean() - 0.5) < 5 * sd / np.sqrt(12)
        for a, b in ((u[:-1], u[1:]), (u[:, :-1], u[:, 1:]), (u[:, :-32], u[:, 32:])):
            assert abs(np.corrcoef(a.ravel(), b.ravel())[0, 1]) < 5 * sd
    a, b = M.fractions(h)
    assert abs(np.corrcoef(a.ravel(), b.ravel())[0, 1]) < 0.01      # they share 12 bits, low ones of the first
    x = np.random.default_rng(0).integers(0, 1 << 32, 1 << 14, dtype=np.uint64).astype(np.uint32)
    y = M.mix(x)
    for i in range(32):
        d = M.mix(x ^ np.uint32(1 << i)) ^ y
        for o in range(32):
            assert abs(((d >> np.uint32(o)) & 1).mean() - 0.5) < 5 * 0.5 / 128
    assert len(np.unique(y)) == len(np.unique(x))
    # chunks of 4096 places have keys of their own
    assert (M.dice(5, 3, [4096])[0] != M.dice(5, 3, [0])[0]) and (M.dice(6, 3, [0])[0] != M.dice(5, 3, [0])[0])


def test_hand_worked_neighbours():
    lo, hi, f, s = M.first_neighbours(group(448.0, 440.0, -9.0, 2.0 ** -9, 1.5 * 2.0 ** -9, 17.0))
    assert s.tolist() == [1.0]
    assert lo[0, :6].tolist() == [448.0, 416.0, 9.0, 2.0 ** -9, 2.0 ** -9, 16.0]
    assert f[0, :6].tolist() == [0.0, 0.75, 0.0, 0.0, 0.5, 0.5] and hi[0, 5] == 18.0
    assert M.first_neighbours(group(448.5))[3].tolist() == [2.0]    # nothing may go past the largest code
    lo, hi, f, s = M.root_neighbours(group(1.9375, 1.03125, 2.0 ** -16, 0.0, 1.0))
    assert s.tolist() == [1.0] and lo[0, :5].tolist() == [1.9375, 1.0, M.LOWEST_ROOT, 0.0, 1.0]
    assert hi[0, 1] == 1.0625 and f[0, 1] == (1.03125 ** 2 - 1) / (1.0625 ** 2 - 1) and f[0, 2] == f[0, 3] == 0.0
    assert M.root_neighbours(group(1.94))[3].tolist() == [2.0]


def test_the_mean_is_kept():
    """Of 2^16 draws; the sum's standard deviation is at most half a code's distance (a square's: of the squares)."""
    n = 1 << 16
    for v in (0.3, 1.0, 3.7e-3, 5e-4):
        x = np.tile(group(1.5, v), n)
        h = M.dice(1, 1, np.arange(x.size))
        got = M.first_stochastic(-x, h).reshape(n, 32)[:, 1]
        lo, hi, _, _ = M.first_neighbours(group(1.5, v))
        assert abs(got.mean() + v) < 5 * (hi[0, 1] - lo[0, 1]) / 2 / 256
        got = M.root_stochastic(x, h).reshape(n, 32)[:, 1] ** 2
        lo, hi, _, _ = M.root_neighbours(group(1.5, v))
        assert abs(got.mean() - v * v) < 5 * (hi[0, 1] ** 2 - lo[0, 1] ** 2) / 2 / 256


def gradients(kind, steps, n, spread, rng):
    fixed = rng.standard_normal(n)
    for t in range(steps):
        g = (fixed if kind == "constant" else rng.standard_normal(n)) * spread
        if kind == "smaller" and t >= steps // 2:
            g = g / 10
        if kind == "gone" and t >= steps // 2:
            g[::2] = 0
        yield g


@pytest.mark.parametrize("beta2", [0.95, 0.999])
@pytest.mark.parametrize("kind", ["constant", "normal", "smaller", "gone"])
def test_moments_follow_the_gradients(kind, beta2):
    """2000 steps beside exact moments.  With codes D apart in v (at most an eighth of it) and a pull of 1 - beta2 back
    to the mean, the roundings leave v a variance of D E|v - mean| / 2, so a standard deviation of at most 1/16 of it
    for a steady v, twice that where v itself moves: the mean of 4096 elements is within 1%, and the median root, which
    is off by half a code (1/32) and half the variance (1/128), within 5%; so is the movement, whose 1/root is off by
    3/8 of the variance and which m's own roundings lengthen by less than that."""
    n, steps, beta1, lr = 4096, 2000, 0.9, 1e-4
    rng = np.random.default_rng(1)
    spread = np.exp(rng.standard_normal(n)) * 1e-3
    m, v, sm, sr, p, sp = (np.zeros(n) for _ in range(6))
    for t, g in enumerate(gradients(kind, steps, n, spread, rng), 1):
        m, v = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
        sm, sv = beta1 * sm + (1 - beta1) * g, beta2 * sr * sr + (1 - beta2) * g * g
        rate, bc2 = lr / (1 - beta1 ** t), 1 - beta2 ** t
        p -= rate * m / (np.sqrt(v / bc2) + 1e-8)
        sp -= rate * sm / (np.sqrt(sv / bc2) + 1e-8)
        h = M.dice(7, t, np.arange(n))
        sm, sr = M.first_stochastic(sm, h), M.root_stochastic(np.sqrt(sv), h)
        assert (sr[sv > 0] > 0).all()
    on = np.arange(n) % 2 == 1 if kind == "gone" else np.ones(n, bool)       # (roots of the others end at code 1)
    ratio = sr[on] / np.sqrt(v[on])
    assert abs(np.median(ratio) - 1) < 0.05
    assert abs((sr[on] ** 2 / spread[on] ** 2).mean() / (v[on] / spread[on] ** 2).mean() - 1) < 0.01
    assert abs(np.abs(sp).mean() / np.abs(p).mean() - 1) < 0.05


def test_rounded_to_nearest_they_do_not():
    """Why: the root of a constant gradient's v, below which half a code is more than a step's move."""
    n, beta2 = 1024, 0.999
    g = np.exp(np.random.default_rng(2).standard_normal(n)) * 1e-3
    v, sr = np.zeros(n), np.zeros(n)
    for _ in range(2000):
        v, sr = beta2 * v + (1 - beta2) * g * g, M.root_nearest(np.sqrt(beta2 * sr * sr + (1 - beta2) * g * g))
    assert np.median(sr / np.sqrt(v)) < 0.5
