"""Rotary positions with one or several position axes (oracle).

The pair (x1, x2) of frequency i turns by θ_i = pos[axis_i]·f_i: (x1 cos θ − x2 sin θ, x2 cos θ + x1 sin θ). Pairs are
(i, i + rot/2) or, adjacent, (2i, 2i + 1); dimensions from rot on pass through.

Test infrastructure only: fp64, as a product of complex numbers.
"""
from __future__ import annotations

import numpy as np


def axis_of(sections, interleaved=False):
    """Axis of every frequency: the sections one after the other, or the axes in turn while their section lasts."""
    if not interleaved:
        return np.repeat(np.arange(len(sections)), sections)
    left, out = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                out.append(a)
                left[a] -= 1
    return np.array(out, np.int64)


def rope(x, pos, axis, freq, adjacent=False, inverse=False):
    """x [N, heads, d] turned; pos [axes, N]; axis, freq [rot/2]."""
    x = np.asarray(x, np.float64)
    theta = np.asarray(pos)[np.asarray(axis)].T.astype(np.float64) * np.asarray(freq, np.float64)  # [N, rot/2]
    half = theta.shape[1]
    i1 = 2 * np.arange(half) if adjacent else np.arange(half)
    i2 = i1 + (1 if adjacent else half)
    z = (x[..., i1] + 1j * x[..., i2]) * np.exp((-1j if inverse else 1j) * theta)[:, None]
    y = x.copy()
    y[..., i1], y[..., i2] = z.real, z.imag
    return y
