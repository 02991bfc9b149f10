"""The rule that AdamW's 8-bit states are rounded by, on the CPU."""
import numpy as np

from oracle import ops_oracle as oo


def test_noise_of_slow_averages_fills_the_interval():
    """Over 4096 seeds a part of 2^-11 at either end is met as often as its size: 1024 of 2^21 numbers, give or take 32
    (and five times that); a byte alone meets neither."""
    z = np.stack([oo.adamw8_noise(512, seed, 0.999) for seed in range(1, 4097)])
    assert z.min() >= 0 and z.max() < 1
    for met in (z < 2.0 ** -11, z >= 1 - 2.0 ** -11):
        assert abs(int(met.sum()) - 1024) < 160
    assert abs(z.mean() - 0.5) < 1e-3


def test_noise_of_other_averages_is_the_byte():
    for beta in (0.0, 0.9, 0.95, 31 / 32):
        assert np.array_equal(oo.adamw8_noise(1000, 7, beta), oo.adamw8_noise(1000, 7))
    assert not np.array_equal(oo.adamw8_noise(1000, 7, 0.97), oo.adamw8_noise(1000, 7))


def test_a_root_that_moves_little_moves():
    """Roots of 1 under zero gradients with beta2 = 0.9999: after 3000 steps 0.8607, the mean of 4096 of them off by 0.01
    at most (their sizes' deviation is below (0.15 / 16)^(1/2) = 0.1, that of the mean 0.0016)."""
    n, beta2 = 4096, 0.9999
    table, r = oo.root_table(), np.ones(n)
    for seed in range(1, 3001):
        z = oo.adamw8_noise(n, seed, beta2)
        r = r * np.sqrt(beta2)
        e = np.ceil(np.log2(r.reshape(-1, 128).max(1) / 248.0)).repeat(128)       # the smallest with r 2^-e <= 248
        u = r * 2.0 ** -e
        lo = np.searchsorted(table, u, side="right") - 1
        up = np.minimum(lo + 1, 255)
        frac = (u - table[lo]) / np.where(up > lo, table[up] - table[lo], 1.0)
        r = table[np.where(frac + z >= 1, up, lo)] * 2.0 ** e
    assert abs(r.mean() / beta2 ** 1500 - 1) < 0.01


def test_large_gradients_count_as_two_to_the_63():
    kw = dict(step=1, lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.1)
    p, g = np.ones(4), np.array([1e20, -3e38, 2.0 ** 63, -1.0])
    got = oo.adamw8_step(p, g, np.zeros(4), np.zeros(4), **kw)
    want = oo.adamw8_step(p, np.clip(g, -2.0 ** 63, 2.0 ** 63), np.zeros(4), np.zeros(4), **kw)
    assert all(np.array_equal(a, b) for a, b in zip(got, want))
    with np.errstate(invalid="ignore"):
        bad = oo.adamw8_step(p, np.array([np.inf, -np.inf, np.nan, 1.0]), np.zeros(4), np.zeros(4), **kw)
    assert not np.isfinite(bad[2][:3]).any() and np.isfinite(bad[2][3])
