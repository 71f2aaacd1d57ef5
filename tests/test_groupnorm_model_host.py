"""A model of group norm's statistics in binary32, thread by thread: it keeps the bounds that
the GPU's results are held to, and does not where a step of the method is left out."""
import numpy as np
import pytest

U = 2.0 ** -24
F, D = np.float32, np.float64


def fma(a, b, c):
    """Binary64 holds the product of two binary32 numbers; the sum's second rounding is of no weight here."""
    return F(D(a) * D(b) + D(c))


def statistics(v, correct=True, recentre=True, base=None):
    """Mean, what its rounding left, and 1/deviation of one group's values v, [threads][rows][vector]: each thread's sums
    about its own shift, moved to their mean after 8, 16, ... rows, then added over the threads."""
    T, R, N = v.shape
    shift = np.zeros(T, F)
    for e in range(N):
        shift = shift + v[:, 0, e]
    shift = shift * F(1 / N)
    s1, s2, past = np.zeros(T, F), np.zeros(T, F), np.zeros(T, F)
    for r in range(1, R + 1):
        for e in range(N):
            d = v[:, r - 1, e] - shift
            s1, s2 = s1 + d, fma(d, d, s2)
        if recentre and 8 <= r < R and r & (r - 1) == 0:
            to = shift + s1 * F(1 / (r * N))
            d = to - shift
            left = fma(-F(r * N), d, s1)
            past, s2 = past + fma(-d, s1 + left, s2), np.zeros(T, F)
            s1, shift = left, to
    s2 = s2 + past
    count, inv = F(R * N), F(1 / (T * R * N))
    about = shift[0] if base is None else F(base)
    m = fma(pairwise(fma(count, shift - about, s1)), inv, about)
    d = m - shift
    dev = fma(-count, d, s1)
    off = F(pairwise(dev) * inv) if correct else F(0)
    var = fma(-off, off, F(pairwise(fma(-d, s1 + dev, s2)) * inv))
    return m, off, F(1) / np.sqrt(max(var, F(1e-30)))


def pairwise(x):
    while len(x) > 1:
        x = x[::2] + x[1::2]
    return x[0]


def errors(v, **kw):
    """Of the mean, in U (deviation + U |mean|), and of 1/deviation, in U."""
    x = v.astype(D)
    mean = x.mean()
    sigma = np.sqrt(((x - mean) ** 2).mean())
    m, off, rstd = statistics(v, **kw)
    return abs(D(m) + D(off) - mean) / (U * (sigma + U * abs(mean))), abs(D(rstd) * sigma - 1) / U


SIZES = [(64, 256, 1), (64, 256, 8), (16, 8, 4), (32, 98, 8), (256, 20, 2)]


def values(size, seed=0):
    return np.random.default_rng(seed).standard_normal(size).astype(F)


@pytest.mark.parametrize("size", SIZES)
def test_bounds_hold(size):
    x = values(size)
    for a in (x, F(1000) + x, F(1e4) + F(1e-3) * x, F(-1e4) + F(1e-2) * x):
        mean, rstd = errors(a)
        assert mean <= 8 and rstd <= 16
    spike, rows = x.copy(), x.copy()
    spike[0, 0, 0] = 1e4
    rows[:3, 0] *= 1e4
    for a in (spike, rows):
        mean, rstd = errors(a)
        assert mean <= 8 and rstd <= 40


def test_without_the_correction_of_the_mean():
    x = values((64, 256, 1))
    assert errors(F(1000) + x, correct=False)[0] > 8
    mean, rstd = errors(F(1e4) + F(1e-3) * x, correct=False)
    assert mean > 8 and rstd > 16


@pytest.mark.parametrize("size", [(64, 256, 1), (64, 256, 8), (32, 98, 8)])
def test_without_moving_the_sums(size):
    x = values(size)
    x[0, 0, 0] = 1e4
    assert errors(x, recentre=False)[1] > 40


def test_about_a_value_of_another_group():
    x = F(1000) + values((64, 256, 1))
    assert errors(x, base=x[0, 0, 0])[1] <= 16
    assert errors(x, base=1e9)[1] > 16
