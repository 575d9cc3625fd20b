"""The clipped policy objective over the tokens of a rollout tree, and its gradients (oracle).

Per token and rollout b through it: min(r·A_b, clip(r, 1 − lo, 1 + hi)·A_b), r = exp(logp − old), where a negative A_b
is multiplied by at most `dual`; minus kl·(e^x − 1 − x), x = ref − logp; plus ent·entropy. The loss is the negative,
weighted and summed. `per_rollout` goes over the rollouts one by one, `objective` over sums of their advantages.

Test infrastructure only: fp64.
"""
from __future__ import annotations

import numpy as np


def _bounded(a, r, lo, hi, dual):
    """The pessimistic value of one advantage, and its slope with respect to log r."""
    plain, cut = r * a, np.clip(r, 1 - lo, 1 + hi) * a
    value = np.minimum(plain, cut)
    slope = np.where(plain <= cut, plain, 0.0)
    if dual is not None:
        floor = np.where(a < 0, dual * a, -np.inf)
        slope = np.where(value >= floor, slope, 0.0)
        value = np.maximum(value, floor)
    return value, slope


def per_rollout(logp, old, advantages, through, lo, hi, dual=None):
    """Σ_b over the rollouts through each token: advantages [B], through [B, N] (0 or 1); (value, slope) [N]."""
    r = np.exp(np.asarray(logp, np.float64) - old)
    value, slope = np.zeros(len(r)), np.zeros(len(r))
    for a, on in zip(advantages, through):
        v, s = _bounded(np.full(len(r), a), r, lo, hi, dual)
        value += on * v
        slope += on * s
    return value, slope


def objective(logp, old, adv, adv_neg=None, ref=None, entropy=None, weights=None, lo=0.2, hi=0.2, dual=None, kl=0.0,
              ent=0.0, g=1.0):
    """(sums [4], dlogp [N], dentropy [N])."""
    logp, old, adv = (np.asarray(t, np.float64) for t in (logp, old, adv))
    w = np.ones(len(logp)) if weights is None else np.asarray(weights, np.float64)
    on = w != 0
    with np.errstate(all="ignore"):
        r = np.exp(logp - old)
        value, slope = _bounded(adv, r, lo, hi, dual)
        if adv_neg is not None:
            v, s = _bounded(-np.asarray(adv_neg, np.float64), r, lo, hi, dual)
            value, slope = value + v, slope + s
        rest = np.zeros(len(logp))
        slope = -slope
        if ref is not None:
            x = np.asarray(ref, np.float64) - logp
            rest = np.expm1(x) - x
            slope = slope - kl * np.expm1(x)
        h = np.zeros(len(logp)) if entropy is None else np.asarray(entropy, np.float64)
        terms = [np.where(on, w * t, 0.0).sum() for t in (-value, rest, h)]
        sums = np.array([terms[0] + kl * terms[1] - ent * terms[2]] + terms)
        return sums, np.where(on, g * w * slope, 0.0), np.where(on, -g * w * ent, 0.0)
