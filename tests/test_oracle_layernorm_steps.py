"""The layer norm oracle's bounds count the steps of the stored type all the way down: values below
float16's normal range, 2^-14, are off by up to 2^-25 however small they are."""
import numpy as np

from oracle import layernorm as ln

HALF, TINY = 2.0 ** -11, 2.0 ** -25


def small_f16(seed, rows, cols):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)).astype(np.float16)
    dy = (2.0 ** -9 * rng.standard_normal((rows, cols))).astype(np.float16)
    gamma = rng.standard_normal(cols).astype(np.float16)
    beta = (2.0 ** -16 * rng.standard_normal(cols)).astype(np.float16)
    return x, dy, gamma, beta


def test_values_rounded_to_f16_are_within_the_bounds():
    """The exact values, rounded once, are off by that rounding alone. A bound that leaves the
    subnormal step out would fail them, and half of that step would too."""
    x, dy, gamma, beta = small_f16(1, 1, 16384)
    y, mean, rstd = ln.forward(x, gamma * 0.0, beta, 1e-5)
    args = (dy, x, mean, rstd, gamma.astype(np.float64))
    off = [np.abs(v.astype(np.float16).astype(np.float64) - v)
           for v in (y, *ln.backward(*args)[:2])]

    def bounds(tiny):
        return (ln.forward_bounds(x, gamma * 0.0, beta, 1e-5, HALF, tiny)[0],
                *ln.backward_bounds(*args, HALF, HALF, tiny, tiny)[:2])

    assert all(np.all(e <= b) for e, b in zip(off, bounds(TINY)))
    assert any(np.any(e > b) for e, b in zip(off[1:], bounds(0.0)[1:]))
    assert any(np.any(e > b) for e, b in zip(off[1:], bounds(TINY / 4)[1:]))


def test_the_step_is_added_once_and_to_its_own_output():
    x, dy, gamma, beta = small_f16(2, 3, 40)
    _, mean, rstd = ln.forward(x, gamma, beta, 1e-5)
    f0, f1 = (ln.forward_bounds(x, gamma, beta, 1e-5, HALF, t) for t in (0.0, TINY))
    assert np.allclose(f1[0] - f0[0], TINY, rtol=1e-6)
    assert np.array_equal(f1[1], f0[1]) and np.array_equal(f1[2], f0[2])
    b0 = ln.backward_bounds(dy, x, mean, rstd, gamma, HALF, HALF)
    b1 = ln.backward_bounds(dy, x, mean, rstd, gamma, HALF, HALF, TINY, 2 * TINY)
    for a, b, t in zip(b0, b1, (TINY, 2 * TINY, 2 * TINY)):
        assert np.allclose(b - a, t, rtol=1e-6)
