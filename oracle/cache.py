"""Operators on the paged cache in float64: plain loops over sequences, heads and
rows, each from its definition.

``K``/``V`` [tokens, Hkv, hd] and ``w`` [tokens, Hkv] are one sequence's
history in token order; query head h reads kv head floor(h * Hkv / Hq).
"""
from __future__ import annotations

import math

import numpy as np


def prompt_attention(q, K, V):
    """q [n, Hq, hd]: the last n positions of K's tokens.  Returns (o [n, Hq, hd],
    lse [Hq, n], weight [tokens, Hkv]: what each token weighs over all rows and
    the heads of its group).  A row before position 0 gives 0 and -inf."""
    n, hq, hd = q.shape
    ctx, hkv = K.shape[:2]
    o, lse = np.zeros((n, hq, hd)), np.full((hq, n), -np.inf)
    weight = np.zeros((ctx, hkv))
    for i in range(n):
        end = ctx - n + i + 1
        if end <= 0:
            continue
        for h in range(hq):
            g = h * hkv // hq
            z = K[:end, g] @ q[i, h] / math.sqrt(hd)
            m = z.max()
            lse[h, i] = m + math.log(np.exp(z - m).sum())
            p = np.exp(z - lse[h, i])
            o[i, h] = p @ V[:end, g]
            weight[:end, g] += p
    return o, lse, weight


def evict_indices(w, keep, recent):
    """Kept tokens [Hkv, min(tokens, keep)] in ascending order: the last `recent`
    and the heaviest of the others; ties go to the lower index, NaN is lightest."""
    n, hkv = w.shape
    if n <= keep:
        return np.tile(np.arange(n), (hkv, 1))
    out = []
    for g in range(hkv):
        order = sorted(range(n - recent), key=lambda t: (bool(np.isnan(w[t, g])), 0.0 if np.isnan(w[t, g]) else -w[t, g], t))
        out.append(sorted(order[: keep - recent]) + list(range(n - recent, n)))
    return np.array(out)
