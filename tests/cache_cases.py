"""Histories for the tests of the cache operators: a paged cache whose unused slots
hold NaN, and the bounds that rounding sets on each result."""
import math

import numpy as np

import oracle


class History:
    """ctxs[s] tokens of every sequence, scattered over shuffled 16-slot blocks."""

    def __init__(self, seed, ctxs, hkv, hd, spare=3, extra_cols=1):
        self.rng = rng = np.random.default_rng(seed)
        self.ctxs, self.hkv, self.hd = ctxs, hkv, hd
        per = max(1, max((c + 15) // 16 for c in ctxs)) + extra_cols
        used = sum((c + 15) // 16 for c in ctxs)
        self.n_blocks = used + spare
        order = rng.permutation(self.n_blocks)
        # entries behind a sequence's tokens are never read: out of range on purpose
        self.table = np.full((len(ctxs), per), 0x7FFFFFF0, dtype=np.int32)
        self.k = np.full((self.n_blocks, hkv, 16, hd), np.nan, dtype=np.float16)
        self.v = self.k.copy()
        self.w = np.full((self.n_blocks, hkv, 16), np.nan, dtype=np.float32)
        self.K, self.V, self.W = [], [], []
        n = 0
        for s, c in enumerate(ctxs):
            K = rng.standard_normal((c, hkv, hd)).astype(np.float16)
            V = rng.standard_normal((c, hkv, hd)).astype(np.float16)
            W = np.abs(rng.standard_normal((c, hkv))).astype(np.float32)
            W[rng.random((c, hkv)) < 0.3] = 0.25   # ties
            for i in range((c + 15) // 16):
                self.table[s, i] = order[n]
                n += 1
            for a, x in ((self.k, K), (self.v, V), (self.w, W)):
                for t in range(c):
                    a[self.table[s, t // 16], :, t % 16] = x[t]
            self.K.append(K)
            self.V.append(V)
            self.W.append(W)

    def gather(self, a, s, n=None, table=None):
        """The first n tokens of sequence s in a paged array."""
        n = self.ctxs[s] if n is None else n
        t = np.arange(n)
        table = self.table if table is None else table
        return a[table[s, t // 16], :, t % 16]

    def owned(self):
        """Which slots hold a token: [n_blocks, 16]."""
        m = np.zeros((self.n_blocks, 16), dtype=bool)
        for s, c in enumerate(self.ctxs):
            t = np.arange(c)
            m[self.table[s, t // 16], t % 16] = True
        return m


# One rounding step, relative: half of torch.finfo(t).eps
U16, U32 = 2.0 ** -11, 2.0 ** -24


def score_error(q, K):
    """Bound of a score's error, per query head: hd products added in fp32 with at most one
    truncation (2 U32) each, the scaling by 1/sqrt(hd) (folded with log2 e or
    not) and the difference to a maximum or log-sum-exp, all relative to the
    sum of the products' magnitudes."""
    hq, hd = q.shape
    hkv = K.shape[1]
    g = np.arange(hq) * hkv // hq
    mag = np.einsum("hd,thd->th", np.abs(q), np.abs(K[:, g]))
    return ((2 * hd + 8) * U32) * mag.max(0) / math.sqrt(hd)


def prompt_reference(h, s, q, ctx=None):
    """The oracle on sequence s's last rows q [n, Hq, hd], with bounds on o (fp16 result,
    probabilities in fp16), lse and weight."""
    K, V = (h.K[s][:ctx].astype(np.float64), h.V[s][:ctx].astype(np.float64))
    q = q.astype(np.float64)
    o, lse, weight = oracle.prompt_attention(q, K, V)
    n, hq, hd = q.shape
    c, hkv = K.shape[:2]
    g = np.arange(hq) * hkv // hq
    bo, bl, bw = np.zeros_like(o), np.zeros_like(lse), np.zeros_like(weight)
    for i in range(n):
        end = c - n + i + 1
        if end <= 0:
            continue
        dz = score_error(q[i], K[:end])
        for a in range(hq):
            z = K[:end, g[a]] @ q[i, a] / math.sqrt(hd)
            p = np.exp(z - lse[a, i])
            # exp (2 U32 and its argument's error), sums of `end` terms, the division
            rel = 2 * dz[a] + (end + 16) * U32 + 4 * U32 * np.abs(z).max()
            absv = np.abs(V[:end, g[a]])
            # p in fp16: U16 relative, 2^-25 absolute below its normal range (the
            # largest p before the division is at least 1); then o in fp16
            bo[i, a] = (U16 + rel) * (p @ absv) + 2.0 ** -25 * absv.sum(0) + U16 * np.abs(o[i, a]) * (1 + U16) + 2.0 ** -25
            bl[a, i] = rel + 4 * U32 * abs(lse[a, i])
            # the weight's exponent has the given lse, rounded to fp32
            bw[:end, g[a]] += p * (rel + 4 * U32 * abs(lse[a, i]))
    bw += weight * (n * hq // hkv + 8) * U32
    return o, lse, weight, bo, bl, bw
