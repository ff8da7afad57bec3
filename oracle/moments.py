"""8-bit moments of an optimizer (oracle): the codes of include/moe_block.h, and
the stochastic rounding of include/moe_moments.h; numpy, float64.

Groups of 32 elements share a power of two, the scale.  m: e4m3 codes; v: its
root as unsigned e4m4 codes without subnormals, code c for (1 + c%16/16) *
2^(c//16 - 15), 0 for 0.  Functions take and return values, not codes: arrays
whose length is a multiple of 32.
"""

from __future__ import annotations

import numpy as np

GROUP = 32
GOLDEN, ROOT2, ROOT3 = 0x9E3779B9, 0x6A09E667, 0xBB67AE85      # 2^32 times the fractions of the golden ratio, and of both roots
LOWEST_ROOT = 17 / 16 * 2.0 ** -15                             # code 1, of scale 1


def mix(x):
    """A bijection of 32-bit numbers whose results' bits all depend on all of x."""
    x = np.asarray(x, np.uint32).copy()
    x ^= x >> np.uint32(16)
    x *= np.uint32(ROOT2)
    x ^= x >> np.uint32(15)
    x *= np.uint32(ROOT3)
    x ^= x >> np.uint32(16)
    return x


def dice(seed: int, t: int, place):
    """The 32 random bits of the elements at `place` in step t: places are counted through a list of tensors, each of
    which begins at a multiple of 4096."""
    place = np.asarray(place, np.uint64)
    chunk, at = (place // np.uint64(4096)).astype(np.uint32), (place % np.uint64(4096)).astype(np.uint32)
    with np.errstate(over="ignore"):
        key = mix(mix(np.uint32((seed + GOLDEN * t) & 0xFFFFFFFF)) + chunk)
        return mix(key + np.uint32(GOLDEN) * at)


def fractions(h):
    """What the two moments' fractions are compared with: the upper 20 bits (m rounds up from the fraction 1 - this on),
    and the lower 24 (a root rounds up where this is below its fraction)."""
    h = np.asarray(h, np.uint32)
    return (h >> np.uint32(12)).astype(np.float64) / 2.0 ** 20, (h & np.uint32(0xFFFFFF)).astype(np.float64) / 2.0 ** 24


def _scale(amax, top):
    """The smallest power of two 2^k, k >= -126, with amax / 2^k <= top, for groups' largest magnitudes."""
    with np.errstate(divide="ignore"):
        m, e = np.frexp(np.where(amax > 0, amax, 1.0))
    mt, et = np.frexp(top)
    k = e - et + (m > mt)
    return np.exp2(np.where(amax > 0, np.maximum(k, -126), -126).astype(np.float64))


def _grid_first(a):
    """The step of e4m3 at magnitudes a."""
    _, e = np.frexp(np.maximum(a, 2.0 ** -6))
    return np.exp2((e - 1 - 3).astype(np.float64))


def first_neighbours(m):
    """The codes' values below and above |m| with stochastic rounding, the fraction of the way between them, the scales."""
    g = np.asarray(m, np.float64).reshape(-1, GROUP)
    s = _scale(np.abs(g).max(1), 448.0)[:, None]
    a = np.abs(g) / s
    step = _grid_first(a)
    lo = np.floor(a / step) * step
    return lo * s, (lo + step) * s, (a - lo) / step, s[:, 0]


def first_stochastic(m, h):
    """m after its rounding with random bits h: its mean is m."""
    lo, hi, f, _ = first_neighbours(m)
    u = fractions(h)[0].reshape(f.shape)
    return (np.where(u >= 1.0 - f, hi, lo) * np.sign(np.asarray(m).reshape(f.shape))).reshape(-1)


def root_neighbours(root):
    """The same of roots, the fraction taken between the codes' squares."""
    r = np.asarray(root, np.float64).reshape(-1, GROUP)
    s = _scale(r.max(1), 1.9375)[:, None]
    a = r / s
    low = a < LOWEST_ROOT
    _, e = np.frexp(np.maximum(a, LOWEST_ROOT))
    step = np.exp2((e - 1 - 4).astype(np.float64))
    lo = np.floor(np.maximum(a, LOWEST_ROOT) / step) * step
    f = (np.maximum(a, LOWEST_ROOT) - lo) * (np.maximum(a, LOWEST_ROOT) + lo) / (step * (2 * lo + step))
    there = r > 0
    return np.where(there, lo, 0.0) * s, np.where(there & ~low, lo + step, np.where(there, lo, 0.0)) * s, np.where(low, 0.0, f), s[:, 0]


def root_stochastic(root, h):
    """Roots after their rounding: the mean of the square is the square, and a root that is not 0 never becomes 0."""
    lo, hi, f, _ = root_neighbours(root)
    u = fractions(h)[1].reshape(f.shape)
    return np.where(u < f, hi, lo).reshape(-1)


def first_nearest(m):
    g = np.asarray(m, np.float64).reshape(-1, GROUP)
    amax = np.abs(g).max(1)
    s = _scale(amax, 448.0)
    s = np.where((amax > 0) & (amax / np.maximum(s / 2, 2.0 ** -126) < 464.0), np.maximum(s / 2, 2.0 ** -126), s)[:, None]
    a = np.abs(g) / s
    step = _grid_first(a)
    return (np.minimum(np.rint(a / step) * step, 448.0) * s * np.sign(g)).reshape(-1)


def root_nearest(root):
    r = np.asarray(root, np.float64).reshape(-1, GROUP)
    amax = r.max(1)
    s = _scale(amax, 1.9375)
    s = np.where((amax > 0) & (amax / np.maximum(s / 2, 2.0 ** -126) < 63 / 32), np.maximum(s / 2, 2.0 ** -126), s)[:, None]
    a = r / s
    _, e = np.frexp(np.maximum(a, LOWEST_ROOT))
    step = np.exp2((e - 1 - 4).astype(np.float64))
    q = np.minimum(np.maximum(np.rint(a / step) * step, LOWEST_ROOT), 1.9375)
    return (np.where(r > 0, q, 0.0) * s).reshape(-1)
