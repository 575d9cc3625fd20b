"""Rotary positions with one or several position axes (oracle).

The pair (x1, x2) of frequency i turns by θ_i = pos[axis_i]·f_i: (x1 cos θ − x2 sin θ, x2 cos θ + x1 sin θ). Pairs are
(i, i + rot/2) or, adjacent, (2i, 2i + 1); dimensions from rot on pass through.

Test infrastructure only: fp64, as a product of complex numbers.
"""
from __future__ import annotations

from fractions import Fraction
from functools import lru_cache

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


_PLACES = 1400


@lru_cache(maxsize=None)
def _digits_of_one_turn():
    """1/2π in units of 2^-_PLACES, from π = 16 atan(1/5) − 4 atan(1/239) in whole numbers."""
    def atan_inv(n):
        term = total = (1 << _PLACES) // n
        k, sign = 1, -1
        while term:
            term //= n * n
            k += 2
            total += sign * (term // k)
            sign = -sign
        return total
    return (1 << (2 * _PLACES - 1)) // (16 * atan_inv(5) - 4 * atan_inv(239))


def angle(pos, freq):
    """pos·freq reduced to less than half a turn (radians), for any int32 position and any double: the product's turns
    are reduced as whole numbers, where a product in fp64 is off by 2^-53 of itself."""
    f = Fraction(float(freq))
    one = 1 << _PLACES
    t = int(pos) * f.numerator * _digits_of_one_turn() // f.denominator % one
    return float(Fraction(t - one if 2 * t >= one else t, one)) * 2.0 * np.pi
