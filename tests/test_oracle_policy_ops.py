"""The oracles of the norm with rotary positions and of the policy objective pinned by hand-derived cases, properties
and differences (CPU)."""
import numpy as np
import pytest

from oracle import decode as D
from oracle import norm_rope as NR
from oracle import policy as P
from oracle import rope as R


def _how(rng, N, axes=1, rot=8, adjacent=False):
    return {"tables": (rng.integers(-50, 50, (axes, N)), rng.integers(0, axes, rot // 2), rng.random(rot // 2)),
            "adjacent": adjacent}


def test_norm_hand_derived():
    x = np.array([[[3.0, 4.0]]])  # mean square 12.5
    np.testing.assert_allclose(NR.forward(x, [2.0, 1.0], 0.0), [[[6 / np.sqrt(12.5), 4 / np.sqrt(12.5)]]], rtol=1e-15)
    assert (NR.forward(np.zeros((1, 1, 2)), None, 1e-6) == 0).all()
    # without eps the result does not depend on the length of x, so dx has no part along x
    dx, _ = NR.backward(np.array([[[1.0, -2.0]]]), x, [2.0, 1.0], 0.0)
    assert abs((dx * x).sum()) < 1e-14


@pytest.mark.parametrize("adjacent", [False, True])
def test_norm_gradients_against_differences(adjacent):
    rng = np.random.default_rng(1)
    x, w, dy = rng.standard_normal((3, 2, 12)), 1 + 0.3 * rng.standard_normal(12), rng.standard_normal((3, 2, 12))
    how = _how(rng, 3, 2, 8, adjacent)
    dx, dw = NR.backward(dy, x, w, 0.1, how)

    def f(x, w):
        return (NR.forward(x, w, 0.1, how) * dy).sum()

    step = 1e-5
    for at in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[at] += step
        b[at] -= step
        assert abs((f(a, w) - f(b, w)) / (2 * step) - dx[at]) < 1e-8
    for j in range(12):
        a, b = w.copy(), w.copy()
        a[j] += step
        b[j] -= step
        assert abs((f(x, a) - f(x, b)) / (2 * step) - dw[j]) < 1e-8


def test_norm_then_rope_is_the_two_in_turn():
    rng = np.random.default_rng(2)
    x, how = rng.standard_normal((4, 3, 16)), _how(rng, 4, 1, 16)
    np.testing.assert_allclose(NR.forward(x, None, 1e-6, how), R.rope(NR.forward(x), *how["tables"]), rtol=1e-15)


def test_two_sums_stand_for_the_rollouts_through_a_token():
    """Σ_b min(r·A_b, clip(r)·A_b) needs Σ A_b over the positive and Σ |A_b| over the negative advantages only."""
    rng = np.random.default_rng(3)
    B, N = 7, 50
    adv = rng.standard_normal(B)
    through = (rng.random((B, N)) < 0.5).astype(float)
    logp, old = -rng.random(N), -rng.random(N)
    for dual in (None, 1.5):
        value, slope = P.per_rollout(logp, old, adv, through, 0.2, 0.3, dual)
        gain, cost = np.maximum(adv, 0) @ through, np.maximum(-adv, 0) @ through
        sums, dlogp, _ = P.objective(logp, old, gain, cost, lo=0.2, hi=0.3, dual=dual)
        np.testing.assert_allclose(sums[1], -value.sum(), rtol=1e-12)
        np.testing.assert_allclose(dlogp, -slope, rtol=1e-12, atol=1e-15)


def test_policy_hand_derived():
    # ratio 1.5 against [0.8, 1.2]: a gain is cut at 1.2 (no slope), a cost is not; ratio 0.5 the other way round
    lr = np.log([1.5, 1.5, 0.5, 0.5])
    sums, dlogp, _ = P.objective(lr, np.zeros(4), np.array([2.0, -2.0, 2.0, -2.0]))
    np.testing.assert_allclose(sums[1], -(2 * 1.2) + 2 * 1.5 - 2 * 0.5 + 2 * 0.8, rtol=1e-14)
    np.testing.assert_allclose(dlogp, [0, 3.0, -1.0, 0], rtol=1e-14)
    # ratio 5: a cost counts dual times
    sums, dlogp, _ = P.objective(np.log([5.0]), [0.0], [-1.0], dual=3.0)
    assert abs(sums[1] - 3.0) < 1e-14 and dlogp[0] == 0
    # the KL term is 0 with slope 0 at the reference, and positive on both sides
    sums, dlogp, _ = P.objective([-1.0, -1.0, -1.0], [-1.0] * 3, np.zeros(3), ref=[-1.0, -0.5, -1.5], kl=2.0)
    assert dlogp[0] == 0 and dlogp[1] < 0 < dlogp[2]
    np.testing.assert_allclose(sums[2], (np.exp(0.5) - 1.5) + (np.exp(-0.5) - 0.5), rtol=1e-14)


def test_policy_gradient_against_differences():
    rng = np.random.default_rng(4)
    N = 40
    logp, old, ref = (-3 * rng.random(N) for _ in range(3))
    gain, cost, w, h = rng.random(N), rng.random(N), rng.integers(0, 3, N) / 2, rng.random(N)
    how = dict(adv_neg=cost, ref=ref, weights=w, lo=0.2, hi=0.28, dual=3.0, kl=0.3, ent=0.1)
    sums, dlogp, dent = P.objective(logp, old, gain, entropy=h, **how)
    step = 1e-6
    r = np.exp(logp - old)
    for t in range(N):
        if min(abs(r[t] - e) for e in (0.8, 1.28, 3.0)) < 1e-4:
            continue  # the slope jumps there
        d = np.zeros(N)
        d[t] = step
        up, down = (P.objective(logp + s, old, gain, entropy=h, **how)[0][0] for s in (d, -d))
        assert abs((up - down) / (2 * step) - dlogp[t]) < 1e-7
        up, down = (P.objective(logp, old, gain, entropy=h + s, **how)[0][0] for s in (d, -d))
        assert abs((up - down) / (2 * step) - dent[t]) < 1e-7


def test_masked_tokens_add_nothing_whatever_they_hold():
    bad = [np.nan, np.inf, -np.inf, 1e30]
    sums, dlogp, dent = P.objective(bad, [0.0] * 4, bad, ref=bad, entropy=bad, weights=[0.0] * 4, kl=1.0, ent=1.0)
    assert (sums == 0).all() and (dlogp == 0).all() and (dent == 0).all()


def test_planted_swap_of_the_clip_sides_is_caught():
    """With the sides of the range swapped for a negative advantage, the hand-derived case fails."""
    lr = np.log([0.5])
    right = P.objective(lr, [0.0], [-2.0])[0][1]
    swapped = 2 * min(0.5, 1.2)  # a cost bounded above instead of below
    assert abs(right - 2 * 0.8) < 1e-14 and abs(swapped - right) > 0.1


def test_decode_hand_derived():
    k = np.array([[[1.0, 0.0]], [[0.0, 1.0]], [[9.0, 9.0]]])
    v = np.array([[[1.0, 2.0]], [[3.0, 4.0]], [[9.0, 9.0]]])
    q = np.array([[[np.log(3.0), 0.0]], [[5.0, 5.0]]])
    O, LSE = D.attention(q, k, v, [(0, 1, 0, 1), (1, 1, 0, 1)], 1.0)  # weights 3/4 and 1/4, over two segments
    np.testing.assert_allclose(O[0, 0], [0.75 * 1 + 0.25 * 3, 0.75 * 2 + 0.25 * 4], rtol=1e-14)
    np.testing.assert_allclose(LSE[0, 0], np.log(4.0), rtol=1e-14)
    assert (O[1] == 0).all() and LSE[0, 1] == -np.inf


def test_decode_is_the_last_row_of_causal_attention_over_a_path():
    from oracle import attention as A
    from oracle import tree as T
    rng = np.random.default_rng(5)
    par, ln = np.array([-1, 0, 0], np.int32), np.array([5, 3, 4], np.int32)
    tab = T.tables(par, ln)
    Q, K, V, dO = (rng.standard_normal((12, h, 8)) for h in (4, 2, 2, 4))
    O, LSE = A.tree_attention_branches(tab, Q, K, V, dO)[:2]
    last = [7, 11]  # the leaves' last tokens
    o, lse = D.attention(Q[last], K, V, [(0, 5, 0, 2), (5, 3, 0, 1), (8, 4, 1, 2)], 8 ** -0.5)
    np.testing.assert_allclose(o, O[last], rtol=1e-12)
    np.testing.assert_allclose(lse, LSE[:, last], rtol=1e-12)
