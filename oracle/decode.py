"""Attention of the next token of running rollouts over the segments that list them (oracle).

Query by query: the key and value rows of its segments put one after the other, one softmax over all of them.

Test infrastructure only: fp64.
"""
from __future__ import annotations

import numpy as np


def attention(q, k, v, segments, scale):
    """q [B, Hq, d]; k, v [rows, Hkv, d]; segments: (kv_begin, kv_len, q_begin, q_end) each. O [B, Hq, d], LSE [Hq, B];
    0 and -inf for a query without keys."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    B, hq, d = q.shape
    hkv = k.shape[1]
    O, LSE = np.zeros((B, hq, d)), np.full((hq, B), -np.inf)
    for b in range(B):
        rows = np.concatenate([np.arange(s, s + n) for s, n, q0, q1 in segments if q0 <= b < q1] + [np.zeros(0, int)])
        rows = rows.astype(int)
        if not len(rows):
            continue
        for h in range(hq):
            s = k[rows, h * hkv // hq] @ q[b, h] * scale
            m = s.max()
            p = np.exp(s - m)
            O[b, h] = p @ v[rows, h * hkv // hq] / p.sum()
            LSE[h, b] = m + np.log(p.sum())
    return O, LSE
