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


# ---- the eight-bit cache: e4m3 codes times a power of two per row

def e4m3_values():
    """The 256 codes' values: sign, four bits of exponent (bias 7), three of fraction; exponent
    0 is subnormal, and all ones (127, 255) is NaN -- there are no infinities."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[c] = math.nan if c & 127 == 127 else -x if c & 128 else x
    return out


def quantize_row(x):
    """One row: (codes uint8 [hd], exponent).  Values that fp16 does not hold become NaN (127)."""
    x = np.asarray(x, dtype=np.float64)
    finite = np.abs(x) < 65520   # false for NaN
    big = np.abs(x[finite]).max(initial=0.0)
    e = -15
    while big > 448 * 2.0 ** e:
        e += 1
    grid = e4m3_values()[:127]   # ascending
    codes = np.full(x.shape, 127, dtype=np.uint8)
    for i in np.flatnonzero(finite):
        y = abs(x[i]) * 2.0 ** -e
        j = min(int(np.searchsorted(grid, y)), 126)
        if j > 0:   # grid[j - 1] < y <= grid[j]: the nearer, of equally near ones the even code
            lo, hi = y - grid[j - 1], grid[j] - y
            if lo < hi or (lo == hi and j % 2 == 1):
                j -= 1
        codes[i] = j + (128 if math.copysign(1.0, x[i]) < 0 else 0)
    return codes, e
