"""Decode attention behind a shared prefix: what it keeps of its probabilities, results within
their own rounding of 64 bits; and scores that are infinite."""
import math

import numpy as np
import pytest

from tests.cache_cases import U16, U32, prompt_reference
from tests.test_gpu_shared_attention import Shared, UNUSED

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from early_exit_decoding_layer_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def set_keys(h, s, t, value):
    """The first component of sequence s's key t, for all kv heads (a shared one for all sequences)."""
    shared = t < h.prefix // 16 * 16
    h.k[h.table[0 if shared else s, t // 16], :, t % 16, 0] = value
    for x in (range(len(h.ctxs)) if shared else [s]):
        if t < h.ctxs[x]:
            h.K[x][t, :, 0] = value


def exact_rows(h, s, q):
    """One row q [Hq, hd] with one component that is not 0, of sequence s, in 64 bits: (o, bound).

    A score is then one product, exact in fp32, times a rounded 1 / sqrt(hd) that may be off by the
    mean of what products of many terms lose (4 U32): 8 U32 of it, twice for a difference.
    Probabilities are two fp16 terms, U16^2 relative, and 2^-25 absolute where the largest is
    2^7 or more.  exp, its sums and the division: U32 for each token, and 64.  The result is rounded
    to fp16: half a step of its binade."""
    K, V = h.K[s].astype(np.float64), h.V[s].astype(np.float64)
    hq, hd = q.shape
    o, bound = np.zeros((hq, hd)), np.zeros((hq, hd))
    for a in range(hq):
        g = a * h.hkv // hq
        z = K[:, g] @ q[a].astype(np.float64) / math.sqrt(hd)
        p = np.exp(z - z.max())
        total, absv = p.sum(), np.abs(V[:, g])
        o[a] = p @ V[:, g] / total
        rel = U16 ** 2 + (16 * np.abs(z).max() + len(z) + 64) * U32
        off = (rel * (p @ absv) + 2.0 ** -32 * absv.sum(0)) / total
        step = np.exp2(np.floor(np.log2(np.maximum(np.abs(o[a]) + off, 2.0 ** -14))) - 11)
        bound[a] = off + step
    return o, bound


CASES = [
    # (query heads, kv heads, hd, prefix, ctxs): own blocks alone; one key tile of 128 rows or
    # fewer; two streams of them; 129 to 256 rows; 512
    (8, 2, 64, 0, [300, 17, 129]), (8, 1, 128, 0, [33, 250]), (8, 2, 64, 64, [64, 80, 65]), (8, 8, 128, 112, [112] * 3),
    (32, 8, 128, 400, [400, 431, 420]), (8, 2, 64, 640, [640, 700, 641]), (8, 1, 64, 300, [304 + i for i in range(20)]),
    (8, 1, 128, 256, [256 + i for i in range(32)]), (8, 1, 128, 144, [144 + i % 40 for i in range(64)]),
]


@pytest.mark.parametrize("faint", [False, True])
@pytest.mark.parametrize("hq,hkv,hd,prefix,ctxs", CASES)
def test_probabilities_keep_their_bits(hq, hkv, hd, prefix, ctxs, faint):
    """Rows whose scores are exact, over values of one sign, so that what a probability loses shows:
    tokens of all weights, or (faint) many tokens of 2^-16 to 2^-20 of the largest."""
    h = Shared(hq + hd + prefix + len(ctxs), ctxs, prefix, hkv, hd)
    q = np.zeros((len(ctxs), hq, hd), dtype=np.float16)
    q[:, :, 0] = h.rng.uniform(0.7, 1.0, (len(ctxs), hq)) * math.sqrt(hd) / 4
    done = set()
    for s, c in enumerate(ctxs):
        for t in range(c):
            at = (0 if t < prefix // 16 * 16 else s, t)
            if at in done:
                continue
            done.add(at)
            # scores of a fourth of these times 0.7 to 1
            x = h.rng.uniform(-64, -48) if faint else h.rng.uniform(-20, 0)
            set_keys(h, s, t, np.float16(0.0 if t == 5 else x))
    for x in [h.v, *h.V]:
        x[...] = np.where(np.isnan(x), x, np.abs(x) + np.float16(0.25))
    assert UNUSED in h.table or prefix == 0
    o = h.call(q, hq).cpu().numpy().astype(np.float64).reshape(q.shape)
    for s in range(len(ctxs)):
        want, bound = exact_rows(h, s, q[s])
        assert np.all(np.abs(o[s] - want) <= bound), (s, np.max(np.abs(o[s] - want) / bound))


# (kv heads, hd, prefix, ctxs): own blocks alone; rows of one tile with one stream and with two;
# 129 to 256 rows, and 512; long own blocks.  Query heads: four to a kv head
INFINITE = [
    (2, 64, 0, [300, 40, 700]), (2, 128, 112, [112, 130, 250, 400]), (2, 64, 640, [640, 900, 655, 1300]),
    (1, 64, 300, [304 + 9 * i for i in range(40)]), (1, 128, 400, [401 + i for i in range(64)]), (2, 128, 64, [3000, 65, 90]),
]


class Without:
    """A history that lacks some tokens of a kv head."""

    def __init__(self, h, s, g, keep):
        self.K, self.V, self.hkv = {s: h.K[s][keep][:, g:g + 1]}, {s: h.V[s][keep][:, g:g + 1]}, 1


def check_infinite(h, q, hit, sign, o):
    """Tokens `hit(s)` have an infinite component 0 in kv head 0's keys, q's is `sign` times a finite one
    or 0: heads with a score of -inf go without them, those with +inf or NaN are NaN."""
    for s, c in enumerate(h.ctxs):
        at = np.zeros(c, dtype=bool)
        at[[t for t in hit(s) if t < c]] = True
        for g in range(h.hkv):
            for a in range(g * 4, g * 4 + 4):
                gone = at if g == 0 else np.zeros_like(at)
                if gone.any() and not sign[a] < 0:
                    assert np.isnan(o[s, a]).all(), (s, a)
                    continue
                if not (~gone).any():
                    assert np.all(o[s, a] == 0), (s, a)
                    continue
                want, _, _, bound, _, _ = prompt_reference(Without(h, s, g, ~gone), s, q[s, a:a + 1][None])
                assert np.all(np.abs(o[s, a] - want[0, 0]) <= bound[0, 0]), (s, a)


@pytest.mark.parametrize("where", ["first", "few", "last of the prefix", "tile", "prefix", "own", "but the last", "all"])
@pytest.mark.parametrize("hkv,hd,prefix,ctxs", INFINITE)
def test_infinite_keys(hkv, hd, prefix, ctxs, where):
    """A score of -infinity weighs nothing, wherever and however many there are (a whole tile, a
    whole part, all of them: then o = 0); one of +infinity makes its row NaN and no other."""
    h = Shared(hd + prefix + len(ctxs), ctxs, prefix, hkv, hd)
    once, most = prefix // 16 * 16, max(ctxs)
    tokens = {
        "first": lambda s: [0], "few": lambda s: [1, once + 1, once + 20, 290, once // 2], "last of the prefix": lambda s: [max(once - 1, 0)],
        "tile": lambda s: range(128, 256), "prefix": lambda s: range(once), "own": lambda s: range(once, most),
        "but the last": lambda s: range(ctxs[s] - 1) if s == 0 else range(once), "all": lambda s: range(most),
    }[where]
    if where == "but the last" and once and once >= ctxs[0]:
        tokens = lambda s: range(once - 1)  # noqa: E731
    q = h.rng.standard_normal((len(ctxs), 4 * hkv, hd)).astype(np.float16)
    sign = np.tile([-1.0, -1.0, 1.0, -1.0], hkv)
    if where == "few":
        sign[0] = 0.0
    q[:, :, 0] = np.abs(q[:, :, 0] + np.float16(0.1)) * sign
    q[:, :, 0] = np.where((q[:, :, 0] == 0) & (sign != 0), sign.astype(np.float16), q[:, :, 0])
    k = h.k.copy()
    for s, c in enumerate(ctxs):
        for t in tokens(s):
            if t < c:
                k[h.table[0 if t < once else s, t // 16], 0, t % 16, 0] = np.inf
    o = h.call(q, 4 * hkv, k=k).cpu().numpy().astype(np.float64).reshape(q.shape)
    check_infinite(h, q, lambda s: [t for t in tokens(s) if t < ctxs[s]], sign, o)
