"""The bounds that the rotation's fp32 results are stored by, on the CPU: its steps in
numpy float32 against 64 bits.

u = 2^-24.  The reduced angle x (|x| <= pi / 4) is rounded once, cos and sin are Taylor series in
z = x x by fused steps, times the factor; a value is fma(a, c, w s).

cos: x is off by half an ulp (0.5 u from 0.5 on), which sin x <= 0.71 passes on: 0.36 u; z by 0.5 u, of
which half arrives: 0.25 u; the series' factor of z (up to 0.5, half an ulp 0.25 u) times z <= 0.62: 0.16 u; the last
sum, below 1: 0.5 u; the rest 0.02 u.  1.3 u together, 0.5 u near x = 0.
sin: x by 0.5 u times cos x <= 0.88: 0.44 u; the series 0.17 u; the last sum 0.5 u: 1.12 u.  Near x = 0, relative to
sin x: x by u, the last sum by u, the series 0.2 u.
factor: u of each.  Product: u of |w s|.  Sum: u of the value, at most |a c| + |w s|.

Of (|a| + |w|) factor: a's share is the error of c, 2 |c| u for factor and sum: 2.7 u at most; w's that of s
and 3 |s| u: 3.6 u (|s| = 0.88).  So 4 u, which leaves room for second orders and for the angle itself.
Of (|a c| + |w s|) factor, where c and s may be small: 2.2 u and 3 u: 5.2 u.  So 5.5 u.
"""
import numpy as np
import pytest

U = 2.0 ** -24
f32, f64 = np.float32, np.float64


def fma(a, b, c):
    """fp32 fused product and sum: the product is exact in fp64 (its sum may round twice, 2^-29 of an ulp)."""
    return (f64(a) * f64(b) + f64(c)).astype(f32)


def series(x):
    """(cos, sin) of fp32 x as the kernel takes them."""
    z = x * x
    s, c = np.full_like(x, 1 / 362880), np.full_like(x, -1 / 3628800)
    for k in (-1 / 5040, 1 / 120, -1 / 6):
        s = fma(s, z, f32(k))
    for k in (1 / 40320, -1 / 720, 1 / 24, -0.5, 1.0):
        c = fma(c, z, f32(k))
    return c, fma(s * z, x, x)


def angles(n, rng):
    """Rests of a quarter turn: spread out, over all powers of two, and next to 0 and the ends."""
    x = np.concatenate([rng.uniform(-1, 1, n) * np.pi / 4, np.pi / 4 * 2.0 ** rng.uniform(-40, 0, n),
                        np.pi / 4 * (1 - 2.0 ** rng.uniform(-30, -3, n)), 0.5 * (1 + rng.uniform(-1, 1, n) * 2.0 ** -10)])
    return np.where(rng.random(x.size) < 0.5, -x, x)


def test_series():
    x = angles(400000, np.random.default_rng(1))
    c, s = series(x.astype(f32))
    assert np.abs(f64(c) - np.cos(x)).max() <= 1.3 * U
    assert np.abs(f64(s) - np.sin(x)).max() <= 1.12 * U
    assert (np.abs(f64(s) - np.sin(x)) / np.abs(np.sin(x))).max() <= 2.2 * U
    assert (np.abs(f64(c) - np.cos(x)) / np.cos(x)).max() <= 2.2 * U


@pytest.mark.parametrize("partner", ["any", "zero", "own zero"])
@pytest.mark.parametrize("factor", [1.0, "any"])
def test_rotated_values(partner, factor):
    rng = np.random.default_rng(2)
    x = angles(400000, rng)
    n = x.size
    f = np.ones(n, f32) if factor == 1.0 else rng.uniform(1, 2, n).astype(f32)
    # 8 significant bits, as of a BF16 value
    a, w = ((rng.integers(128, 256, n) * 2.0 ** rng.integers(-12, 4, n) * rng.choice([-1, 1], n)).astype(f32) for _ in range(2))
    if partner == "zero":
        w[:] = 0
    elif partner == "own zero":
        a[:] = 0
    c, s = series(x.astype(f32))
    tc, ts = np.cos(x), np.sin(x)
    for c, s, tc, ts in ((c, s, tc, ts), (s, c, ts, tc)):          # an odd quarter turn exchanges them
        got = f64(fma(a, c * f, w * (s * f)))
        want = (f64(a) * tc + f64(w) * ts) * f64(f)
        err = np.abs(got - want)
        assert (err / ((np.abs(f64(a)) + np.abs(f64(w))) * f64(f))).max() <= 4 * U
        assert (err / ((np.abs(a * tc) + np.abs(w * ts)) * f64(f))).max() <= 5.5 * U


def test_quotients_of_8_bits():
    """The bounds' ends contain the quotient by a scale: q - room and q + room in fp32, room = 2^-21 (size / scale + |q|)."""
    rng = np.random.default_rng(3)
    x = angles(400000, rng)
    n = x.size
    f, scale = rng.uniform(1, 2, n).astype(f32), rng.uniform(0.25, 4, n).astype(f32)
    a, w = (rng.integers(-255, 256, n).astype(f32) for _ in range(2))
    a[::3], w[1::3] = 0, 0
    c, s = series(x.astype(f32))
    c, s = c * f, s * f
    y = fma(a, c, w * s)
    size = fma(np.abs(a), np.abs(c), np.abs(w * s))
    inv = f32(1) / scale
    q = y * inv
    room = fma(size, inv, np.abs(q)) * f32(2.0 ** -21)
    want = (f64(a) * np.cos(x) + f64(w) * np.sin(x)) * f64(f) / f64(scale)
    assert np.all(f64(q - room) <= want) and np.all(want <= f64(q + room))
    # values that do not turn: y itself
    q = a * inv
    room = q * f32(2.0 ** -21)
    want = f64(a) / f64(scale)
    lo, hi = np.minimum(q - room, q + room), np.maximum(q - room, q + room)
    assert np.all(f64(lo) <= want) and np.all(want <= f64(hi))
