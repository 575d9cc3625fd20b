"""Log-prob of given tokens, entropy and top alternatives per row of logits, and the gradient of a function of
them (oracle).

Definitions, with p = softmax(z) of a row: logp = log p_y, entropy = −Σ_v p_v log p_v (0·log 0 = 0), the top
alternatives are the k largest logits in descending order with ties to the lower index. A masked logit (−inf) has
p = 0. A row with nothing but −inf has no distribution: lse = logp = −inf, entropy 0, gradient 0 (the reading of the
library; the formulas leave it open).

Test infrastructure only. fp64 throughout, on the exact values the GPU receives.
"""
from __future__ import annotations

import numpy as np


def _log_p(z):
    """lse, log p = (z − max) − log Σ e^(z − max) (so that it holds at any size of z), rows without distribution."""
    m = z.max(axis=1, keepdims=True)
    empty = np.isneginf(m[:, 0])
    d = z - np.where(empty[:, None], 0.0, m)
    with np.errstate(divide="ignore"):
        log_s = np.log(np.exp(d).sum(axis=1))
    lp = np.where(empty[:, None], -np.inf, d - np.where(empty, 0.0, log_s)[:, None])
    return np.where(empty, -np.inf, m[:, 0] + log_s), lp, empty


def token_logprob(z, y=None, k=0):
    """logp [N] (None without y), entropy [N], lse [N], top_ids [N, k], top_logp [N, k] of logits z [N, V]."""
    z = np.asarray(z, np.float64)
    lse, lp, empty = _log_p(z)
    p = np.exp(lp)
    entropy = -(p * np.where(p > 0, lp, 0.0)).sum(axis=1)
    logp = None if y is None else lp[np.arange(len(z)), np.asarray(y, np.int64)]
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k]
    return logp, np.where(empty, 0.0, entropy), lse, ids, np.take_along_axis(lp, ids, axis=1)


def token_logprob_grad(z, y=None, dlogp=None, dentropy=None, dlse=None, top_ids=None, dtop=None):
    """d/dz of Σ dlogp·logp + dentropy·entropy + dlse·lse + Σ_j dtop_j·(z − lse)[top_ids_j] (each term optional)."""
    z = np.asarray(z, np.float64)
    N = len(z)
    _, lp, empty = _log_p(z)
    p = np.exp(lp)
    lp = np.where(p > 0, lp, 0.0)
    rows = np.arange(N)
    dz = np.zeros_like(z)
    if dlogp is not None:
        dz -= p * np.asarray(dlogp, np.float64)[:, None]
        np.add.at(dz, (rows, np.asarray(y, np.int64)), np.asarray(dlogp, np.float64))
    if dentropy is not None:
        h = -(p * lp).sum(axis=1, keepdims=True)
        dz -= p * (lp + h) * np.asarray(dentropy, np.float64)[:, None]
    if dlse is not None:
        dz += p * np.asarray(dlse, np.float64)[:, None]
    if dtop is not None:
        g = np.asarray(dtop, np.float64)
        dz -= p * g.sum(axis=1, keepdims=True)
        np.add.at(dz, (rows[:, None], np.asarray(top_ids, np.int64)), g)
    dz[empty] = 0.0
    return dz
