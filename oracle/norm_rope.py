"""RMS norm of every head with the rotary positions behind it, and its gradients (oracle).

n = w·x/size with size = (mean x² + eps)^1/2 over the head, y = R(pos)·n. The gradient of the norm is the projection
of w·g/size (g = R(−pos)·dy) off the direction of x, up to eps.

Test infrastructure only: fp64.
"""
from __future__ import annotations

import numpy as np

from oracle import rope as R


def _turn(x, how, inverse=False):
    return R.rope(x, *how["tables"], how.get("adjacent", False), inverse) if how else x


def forward(x, w=None, eps=1e-6, how=None):
    """x [N, heads, d], w [d]; how: {"tables": (pos, axis, freq), "adjacent"} of oracle.rope, None = no rotation."""
    x = np.asarray(x, np.float64)
    n = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    return _turn(n if w is None else n * np.asarray(w, np.float64), how)


def backward(dy, x, w=None, eps=1e-6, how=None):
    """(dx, dw) of forward."""
    x = np.asarray(x, np.float64)
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, np.float64)
    size = np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    g = _turn(np.asarray(dy, np.float64), how, True)
    unit = x / size
    dx = (g * w - unit * (g * w * unit).mean(-1, keepdims=True)) / size
    return dx, (g * unit).sum((0, 1))
