"""The oracles of the per-token operators pinned by hand-derived cases, properties and differences (CPU)."""
import numpy as np
import pytest

from oracle import rope as R
from oracle import token_logprob as TL


def test_hand_derived_rows():
    z = np.array(
        [[0.0, np.log(2.0), 0.0, np.log(4.0)], [5.0, 5.0, 5.0, 5.0], [np.log(3.0), 0.0, -np.inf, -np.inf]])
    logp, h, lse, ids, top = TL.token_logprob(z, [1, 2, 0], 3)
    np.testing.assert_allclose(logp, np.log([2 / 8, 1 / 4, 3 / 4]), rtol=1e-14)
    p0 = np.array([1, 2, 1, 4]) / 8
    np.testing.assert_allclose(h, [-(p0 * np.log(p0)).sum(), np.log(4), 0.75 * np.log(4 / 3) + 0.25 * np.log(4)],
                               rtol=1e-14)
    np.testing.assert_allclose(lse, [np.log(8), 5 + np.log(4), np.log(4)], rtol=1e-14)
    assert ids.tolist() == [[3, 1, 0], [0, 1, 2], [0, 1, 2]]
    np.testing.assert_allclose(top[0], np.log([4 / 8, 2 / 8, 1 / 8]), rtol=1e-14)
    assert top[2, 2] == -np.inf


def test_row_without_distribution():
    z = np.full((1, 3), -np.inf)
    logp, h, lse, ids, top = TL.token_logprob(z, [1], 2)
    assert logp[0] == lse[0] == -np.inf and h[0] == 0 and ids.tolist() == [[0, 1]] and (top == -np.inf).all()
    assert (TL.token_logprob_grad(z, [1], np.ones(1), np.ones(1), np.ones(1)) == 0).all()


@pytest.mark.parametrize("masked", [False, True])
def test_gradient_against_differences(masked):
    rng = np.random.default_rng(3)
    N, V, k = 4, 11, 3
    z = rng.standard_normal((N, V)) * 2
    if masked:
        z[:, [2, 7]] = -np.inf
    y = np.array([0, 1, 3, 10])
    ids = np.array([[0, 1, 0], [3, 3, 3], [4, 5, 6], [10, 9, 8]])  # repeated ids, and the target among them
    dl, dh, ds, dt = rng.standard_normal(N), rng.standard_normal(N), rng.standard_normal(N), rng.standard_normal((N, k))

    def objective(z):
        logp, h, lse, _, _ = TL.token_logprob(z, y)
        lp = z - lse[:, None]
        return (dl * logp + dh * h + ds * lse).sum() + (dt * np.take_along_axis(lp, ids, axis=1)).sum()

    g = TL.token_logprob_grad(z, y, dl, dh, ds, ids, dt)
    step = 1e-5
    for t in range(N):
        for v in range(V):
            if z[t, v] == -np.inf:
                assert g[t, v] == 0
                continue
            a, b = z.copy(), z.copy()
            a[t, v] += step
            b[t, v] -= step
            assert abs((objective(a) - objective(b)) / (2 * step) - g[t, v]) < 1e-8  # step^2 and 1e-15/step


def test_planted_sign_of_the_entropy_term_is_caught():
    """The gradient of the entropy sums to 0 over a row and falls on the likely tokens; a flipped sign fails both
    the differences above and this property."""
    z = np.array([[2.0, 0.0, 0.0]])
    g = TL.token_logprob_grad(z, dentropy=np.ones(1))
    assert abs(g.sum()) < 1e-15 and g[0, 0] < 0 < g[0, 1]


def test_axis_maps():
    assert R.axis_of((2, 1, 1)).tolist() == [0, 0, 1, 2]
    assert R.axis_of((3, 1, 2), interleaved=True).tolist() == [0, 1, 2, 0, 2, 0]


@pytest.mark.parametrize("adjacent", [False, True])
def test_rotation_properties(adjacent):
    rng = np.random.default_rng(0)
    N, d, rot = 6, 16, 12
    axis, freq = R.axis_of((3, 2, 1)), 10000.0 ** (-np.arange(6) / 6)
    pos = rng.integers(-50, 50, (3, N))
    x, y = rng.standard_normal((2, N, 2, d))
    a, b = R.rope(x, pos, axis, freq, adjacent), R.rope(y, pos, axis, freq, adjacent)
    np.testing.assert_allclose((a * b).sum(-1), (x * y).sum(-1), atol=1e-12)     # orthogonal: the inverse is the VJP
    np.testing.assert_allclose(R.rope(a, pos, axis, freq, adjacent, inverse=True), x, atol=1e-12)
    assert (a[..., rot:] == x[..., rot:]).all()
    # scores depend on differences of positions only
    s0 = (R.rope(x, pos, axis, freq, adjacent) * R.rope(y, pos + 3, axis, freq, adjacent)).sum(-1)
    s1 = (R.rope(x, pos + 7, axis, freq, adjacent) * R.rope(y, pos + 10, axis, freq, adjacent)).sum(-1)
    np.testing.assert_allclose(s0, s1, atol=1e-12)
    # one frequency, one quarter turn, by hand
    q = R.rope(np.array([[[1.0, 2.0]]]), np.array([[1]]), [0], [np.pi / 2], adjacent)
    np.testing.assert_allclose(q, [[[-2.0, 1.0]]], atol=1e-15)


def test_angles_reduced_in_whole_numbers():
    """Against fp64 where its product is exact enough, and by doubling and adding angles where it is not."""
    for p in (0, 1, -5, 1000):
        for f in (1.0, 0.25, -3.5, 1e-4):
            d = R.angle(p, f) - p * f
            assert abs(d - 2 * np.pi * round(d / (2 * np.pi))) < 1e-12
    assert abs(R.angle(1, 2 * np.pi) + 2.4492935982947064e-16) < 1e-30  # 2π as a double is below 2π by this much
    # doubling the frequency doubles the angle, at any size
    for f in (7.0, 1e17, 1e300):
        d = R.angle(1, 2 * f) - 2 * R.angle(1, f)
        assert abs(d - 2 * np.pi * round(d / (2 * np.pi))) < 1e-14
    # two positions' angles add up
    d = R.angle(2 ** 31 - 1, 7.0) - (R.angle(2 ** 30, 7.0) + R.angle(2 ** 30 - 1, 7.0))
    assert abs(d - 2 * np.pi * round(d / (2 * np.pi))) < 1e-14
