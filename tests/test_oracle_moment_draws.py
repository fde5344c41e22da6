"""The drawn codes of a second moment in 8 bits, in the oracle: each draw is one of the two codes about the value, its
mean is the value, and a running average kept in them follows the exact one over thousands of steps, where one kept in
the nearest codes stops.  The words against the scalar definition of the generator.

Bounds.  An average a of squares kept in drawn codes is off by e <- beta2 e + x, x of mean 0 between -D and D for
neighbours D apart, so of a variance of D^2 / 4 at most; the bound sums these beside the run and takes five of their
roots, over all elements of a part of the block at once, and 1e-3 of the sum for the rounding of the steps (2^-24 a
step, over 1 / (1 - beta2) steps).
"""

import numpy as np
import pytest

from oracle import experts_oracle as X
from oracle import qlora_oracle as O

B2 = 0.999


def test_words():
    for seed, step, chunk, count in ((0, 1, 0, 9), (2 ** 63 + 12345, 7, 3, 130), (5, 2 ** 31 + 3, 2 ** 24 - 2, 4)):
        got = X.moment8_draws(seed, step, chunk, count)
        for i in range(count):
            c = (2 ** 33 * step + 512 * chunk + i // 4) % 2 ** 64
            want = O.philox4x32_10((c & 0xFFFFFFFF, c >> 32, 0, 0), (seed & 0xFFFFFFFF, seed >> 32))[i % 4]
            assert int(got[i]) == want


def test_codes_about_the_value():
    rng = np.random.default_rng(3)
    v = (rng.standard_normal(1000) * 10.0 ** rng.uniform(-4, 2, 1000)) ** 2
    v[::19] = 0.0
    v[128:256] = 0.0
    codes, steps = X.moment8_pack_drawn(v, rng.integers(0, 2 ** 32, 1000, dtype=np.uint64))
    near, same = X.moment8_pack(v, False)
    assert np.array_equal(steps, same) and np.array_equal(codes == 0, v == 0) and not codes[128:256].any()
    assert np.abs(codes.astype(int) - near).max() == 1
    d, k = np.repeat(steps.astype(np.float64), 128)[:1000], codes.astype(np.float64)
    up, down = ((k + 1) ** 2 * d) ** 2, (np.maximum(k - 1, 0) ** 2 * d) ** 2
    assert np.all((down <= v * (1 + 1e-12)) & ((v < up) | (d == 0) | (k == 255)))


def test_mean():
    """20000 draws of each of 128 values: the mean is off by five times its own spread at most."""
    rng = np.random.default_rng(4)
    v = rng.uniform(0.2, 1.0, 128) ** 2
    v[0] = 1.1
    n, total = 20000, np.zeros(128)
    for _ in range(n):
        codes, steps = X.moment8_pack_drawn(v, rng.integers(0, 2 ** 32, 128, dtype=np.uint64))
        total += X.moment8_values(codes, steps, False)
    k, d = codes.astype(np.float64), float(steps[0])
    apart = ((k + 2) ** 2 * d) ** 2 - ((k + 1) ** 2 * d) ** 2
    off = np.abs(total / n - v)[1:]  # the first is the largest, whose code is 255
    assert np.all(off <= 5 * apart[1:] / 2 / np.sqrt(n))


def follow(pack, scale, steps):
    """(exact averages, kept ones, variance bounds) after `steps` steps of gradients of `scale(step)`."""
    rng = np.random.default_rng(6)
    n = 512
    v, kept, var = np.zeros(n), np.zeros(n), np.zeros(n)
    for t in range(1, steps + 1):
        g2 = (rng.standard_normal(n) * scale(t)) ** 2
        v = B2 * v + (1 - B2) * g2
        codes, d = pack(B2 * kept + (1 - B2) * g2, t)
        kept = X.moment8_values(codes, d, False)
        k, d = codes.astype(np.float64), np.repeat(d.astype(np.float64), 128)
        var = B2 ** 2 * var + (((k + 1) ** 2 * d) ** 2 - (np.maximum(k - 1, 0) ** 2 * d) ** 2) ** 2 / 4
    return v, kept, var


@pytest.mark.parametrize("change", [1.0, 0.2, 2.0])
def test_the_average_follows(change):
    """Gradients of every other element change by a factor after 1500 steps."""
    odd = np.arange(512) % 2 == 1
    scale = lambda t: np.where(odd & (t > 1500), change, 1.0)
    v, kept, var = follow(lambda x, t: X.moment8_pack_drawn(x, X.moment8_draws(9, t, 0, 512)), scale, 4500)
    for part in (odd, ~odd):
        assert abs((kept - v)[part].sum()) <= 5 * np.sqrt(var[part].sum()) + 1e-3 * v[part].sum()
    if change == 0.2:  # what the nearest codes do: the roots stay where they were
        v, kept, _ = follow(lambda x, t: X.moment8_pack(x, False), scale, 4500)
        assert np.median(np.sqrt(kept / v)[odd]) > 2.0
