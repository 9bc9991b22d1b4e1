"""Histories in the eight-bit cache for its tests, whose unused slots hold NaN codes and
extreme exponents, and the bounds that rounding sets on the attention over them."""
import math

import numpy as np

import oracle
from tests.cache_cases import U16, U32, score_error

VALUES = oracle.e4m3_values()
UNUSED = 0x7FFFFFF0   # in block tables: entries that are never read


class EightBit:
    """ctxs[s] tokens of every sequence over shuffled blocks; codes of all sizes, exponents
    about `scale`."""

    def __init__(self, seed, ctxs, hkv, hd, spare=3, extra_cols=1, scale=-8, spread=2):
        self.rng = rng = np.random.default_rng(seed)
        self.ctxs, self.hkv, self.hd = ctxs, hkv, hd
        per = max(1, max((c + 15) // 16 for c in ctxs)) + extra_cols
        self.n_blocks = sum((c + 15) // 16 for c in ctxs) + spare
        order = rng.permutation(self.n_blocks)
        self.table = np.full((len(ctxs), per), UNUSED, dtype=np.int32)
        self.codes = np.full((self.n_blocks, hkv, 2, 16, hd), 0x7F, dtype=np.uint8)
        self.exps = rng.choice(np.array([-128, 127], dtype=np.int8), (self.n_blocks, hkv, 2, 16))
        n = 0
        for s, c in enumerate(ctxs):
            nb = (c + 15) // 16
            self.table[s, :nb] = order[n:n + nb]
            n += nb
            t = np.arange(c)
            # normal values, as a quantised row holds them: up to 448, most far below
            x = rng.standard_normal((c, hkv, 2, hd)) * 100
            codes = np.searchsorted(VALUES[:127], np.minimum(np.abs(x), 440)).astype(np.uint8)
            self.codes[self.table[s, t // 16], :, :, t % 16] = codes + 128 * (x < 0)
            self.exps[self.table[s, t // 16], :, :, t % 16] = rng.integers(scale - spread, scale + spread + 1, (c, hkv, 2))

    def history(self, s, codes=None):
        """(K, V) of sequence s: [tokens, Hkv, hd] in 64 bits, and V's exponents [tokens, Hkv]."""
        t = np.arange(self.ctxs[s])
        at = self.table[s, t // 16], slice(None), slice(None), t % 16
        e = self.exps[at].astype(np.float64)
        x = VALUES[(self.codes if codes is None else codes)[at]] * np.exp2(e)[..., None]
        return x[:, :, 0], x[:, :, 1], e[:, :, 1]


def attention_reference(q, K, V, ev):
    """One row q [Hq, hd] over K, V: (o, its error's bound) in 64 bits."""
    hq, hd = q.shape
    c, hkv = K.shape[:2]
    o, bound = np.zeros((hq, hd)), np.zeros((hq, hd))
    if c == 0:
        return o, bound
    dz = score_error(q, K)
    for h in range(hq):
        g = h * hkv // hq
        z = K[:, g] @ q[h] / math.sqrt(hd)
        p = np.exp(z - z.max())
        total = p.sum()
        o[h] = p @ V[:, g] / total
        # q is exact down to 2^-27 of its largest value (parts of four bits, 2^-5 apart)
        dq = 2.0 ** -27 * np.abs(q[h]).max() * np.abs(K[:, g]).sum(1).max() / math.sqrt(hd)
        rel = 2 * (dz[h] + dq) + (c + 32) * U32 + 4 * U32 * np.abs(z).max()
        # probabilities with V's scale, x = p 2^e: 2^-12 relative, 2^-24 of the largest absolute
        x = p * np.exp2(ev[:, g])
        absv = np.abs(V[:, g])
        bound[h] = ((2.0 ** -12 + rel) * (p @ absv) + 2.0 ** -24 * x.max() * (absv / np.exp2(ev[:, g])[:, None]).sum(0)) / total
        bound[h] += U16 * (np.abs(o[h]) + bound[h]) + 2.0 ** -25
    return o, bound
