"""What decode attention behind a shared prefix keeps of its probabilities: results within
their own rounding of 64 bits."""
import math

import numpy as np
import pytest

from tests.cache_cases import U16, U32
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
