"""The eight-bit cache: every rounding that writing makes, against a search of the table of codes;
what decode attention over it keeps of its probabilities; queries and values of very
different size."""
import math

import numpy as np
import pytest

import oracle
from tests.cache_cases import U32
from tests.quantized_cases import VALUES, EightBit, attention_reference
from tests.test_gpu_cache_ops import dev
from tests.test_gpu_quantized_cache import check_decode

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import early_exit_decoding_layer_gb300 as ee  # noqa: E402

GRID = VALUES[:127]   # the codes' values from 0 to 448


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from early_exit_decoding_layer_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def quantized(x):
    """oracle.quantize_row for all rows at once."""
    x = np.asarray(x, dtype=np.float64)
    held = np.abs(x) < 65520
    y = np.where(held, np.abs(x), 0.0)
    e = np.full(len(x), -15)
    for k in range(-15, 8):
        e += y.max(1) > 448 * 2.0 ** k
    y = y * np.exp2(-e.astype(np.float64))[:, None]
    j = np.minimum(np.searchsorted(GRID, y), 126)
    lo, hi = y - GRID[np.maximum(j - 1, 0)], GRID[j] - y
    j = np.where((j > 0) & ((lo < hi) | ((lo == hi) & (j % 2 == 1))), j - 1, j)
    return np.where(held, j + np.where(np.signbit(x), 128, 0), 127).astype(np.uint8), e.astype(np.int8)


def filled(largest, values):
    """Rows of 64: `largest`, then 63 of `values`, which are no larger."""
    v = np.concatenate([values, np.zeros(-len(values) % 63, values.dtype)]).reshape(-1, 63)
    return np.concatenate([np.full((len(v), 1), largest, values.dtype), v], 1)


def halves():
    """All fp16 values in rows of all exponents, with the largest and least maximum of each."""
    x = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16).view(np.float16)
    x = x[np.isfinite(x)]
    size = np.unique(np.abs(x).astype(np.float64))
    out, last = [], 0.0
    for e in range(-15, 9):
        fits = size[size <= 448 * 2.0 ** e]
        top = fits[-1] if e < 8 else 65504.0
        above = size[size > last][0]   # the least value that the exponent before does not hold
        for big, some in ((above, x), (top, x)) if e in (-15, 0, 8) else ((top, x), (above, x[::7])):
            out.append(filled(np.float16(big), some[np.abs(some.astype(np.float64)) <= big]))
        last = top
    return np.concatenate(out)


def singles():
    """Every border between two codes at every exponent, and its neighbours in fp32, with both signs."""
    mid = ((GRID[:-1] + GRID[1:]) / 2).astype(np.float32)
    border = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9)), GRID.astype(np.float32)])
    out = []
    for e in range(-15, 9):
        scale = np.float32(2.0 ** e)
        v = np.concatenate([border, -border]) * scale
        v = v[np.abs(v) < 65520]
        # a maximum above the last exponent's 448, below this one's
        top = np.float32(min(448 * 2.0 ** e, 65519.99))
        out.append(filled(top, v[np.abs(v) <= top]))
        if e > -15:
            low = np.nextafter(np.float32(448 * 2.0 ** (e - 1)), np.float32(1e9))
            out.append(filled(low, v[np.abs(v) <= low]))
            out.append(filled(np.float32(448 * 2.0 ** (e - 1)), v[np.abs(v) <= 448 * 2.0 ** (e - 1)]))
    odd = np.array([0.0, -0.0, 1e-45, -1e-40, 1e-38, 65519.99, 65520.0, -65520.0, 1e30, np.inf, -np.inf, np.nan, 1.0], np.float32)
    out += [filled(np.float32(0.0), odd[:5]), filled(np.float32(np.nan), odd), filled(np.float32(1e30), odd[:5])]
    return np.concatenate(out)


@pytest.mark.parametrize("make", [halves, singles])
def test_every_rounding(make):
    rows = make()
    want, exponent = quantized(rows)
    for i in range(0, len(rows), 401):   # the two forms of the oracle
        codes, e = oracle.quantize_row(rows[i])
        assert np.array_equal(codes, want[i]) and e == exponent[i], i
    assert set(exponent) == set(range(-15, 9))
    per, T = 16384, len(rows)
    S = (T + per - 1) // per
    nb = S * per // 16
    codes = torch.zeros(nb, 1, 2, 16, 64, dtype=torch.uint8, device="cuda")
    exps = torch.zeros(nb, 1, 2, 16, dtype=torch.int8, device="cuda")
    cu = np.minimum(np.arange(S + 1) * per, T).astype(np.int32)
    k, v = dev(rows), dev(np.ascontiguousarray(rows[::-1]))
    ee.quantize_cache(k, v, codes, exps, torch.arange(nb, dtype=torch.int32, device="cuda").view(S, -1), dev(cu), dev(np.diff(cu)), per)
    codes, exps = codes.cpu().numpy(), exps.cpu().numpy()
    for kv in range(2):
        got, e = codes[:, 0, kv].reshape(-1, 64)[:T], exps[:, 0, kv].reshape(-1)[:T]
        w, we = (want, exponent) if kv == 0 else (want[::-1], exponent[::-1])
        assert np.array_equal(e, we)
        nan = (got & 127) == 127
        assert np.array_equal(nan, (w & 127) == 127) and np.array_equal(got[~nan], w[~nan])


def test_small_components_beside_a_large_one():
    """A query's components that are 2^-14 of its largest one, which meets keys of 0: all three of the
    parts that a component goes in as count."""
    hd, n = 64, 404
    # 224 for the largest one; 2^-7 + 2^-11 + 2^-14 + 2^-17, whose parts of four bits are 2^-7,
    # 2^-6 + 2^-9 times 2^-5 and 2^-7 times 2^-10
    big, small = 57344.0, 2.0 + 2.0 ** -3 + 2.0 ** -6 + 2.0 ** -9
    assert float(np.float16(small)) == small
    h = EightBit(3, [n], 2, hd)
    t = np.arange(n)
    at = h.table[0, t // 16], slice(None), slice(None), t % 16
    codes, exps = h.codes[at], h.exps[at]   # [n, kv heads, 2, hd]
    # scores of 3 for the first token and of -3 for the others, whose values are -1 to its 1: o is
    # about 0, and moves by half of what a score does
    one = int(np.searchsorted(GRID, 0.1875))
    codes[:, :, 0] = one + 128 * (t > 0)[:, None, None]
    codes[:, :, 0, 0] = 0
    codes[:, :, 1] = int(np.searchsorted(GRID, 1.0)) + 128 * (t > 0)[:, None, None]
    exps[:] = 0
    h.codes[at], h.exps[at] = codes, exps
    q = np.full((1, 4, hd), small, dtype=np.float16)
    q[:, :, 0] = big
    check_decode(h, q, 4)
    K, V, ev = h.history(0)
    want, bound = attention_reference(q[0].astype(np.float64), K, V, ev)
    two = q[0].astype(np.float64)
    two[:, 1:] -= 2.0 ** -9   # without the third parts the check would not pass
    without, _ = attention_reference(two, K, V, ev)
    assert np.all(np.abs(without - want) > bound)


def exact_rows(q, K, V, ev):
    """One row q [Hq, hd] with one component that is not 0, in 64 bits: (o, bound).

    A score is then one product, exact in fp32, times a rounded log2 e / sqrt(hd) and plus V's exponent:
    4 U32 of it, twice for a difference.  Probabilities with V's scale, x = p 2^e, go in as four parts:
    2^-19 of each, and 2^-29 of the largest.  exp, sums and the division: U32 for each token, and 64.
    The result is rounded to fp16: half a step of its binade."""
    hq, hd = q.shape
    o, bound = np.zeros((hq, hd)), np.zeros((hq, hd))
    for a in range(hq):
        g = a * K.shape[1] // hq
        z = K[:, g] @ q[a] / math.sqrt(hd)
        p = np.exp(z - z.max())
        x, absv, total = p * np.exp2(ev[:, g]), np.abs(V[:, g]), p.sum()
        o[a] = p @ V[:, g] / total
        rel = 2.0 ** -19 + (8 * np.abs(z).max() + 8 * np.abs(ev).max() + len(z) + 64) * U32
        off = (rel * (p @ absv) + 2.0 ** -29 * x.max() * (absv / np.exp2(ev[:, g])[:, None]).sum(0)) / total
        bound[a] = off + np.exp2(np.floor(np.log2(np.maximum(np.abs(o[a]) + off, 2.0 ** -14))) - 11)
    return o, bound


def check_exact(h, q, hq, max_ctx):
    B = len(h.ctxs)
    o = ee.quantized_attention(dev(q.reshape(B, -1)), dev(h.codes), dev(h.exps), dev(h.table), dev(np.array(h.ctxs, np.int32) - 1), hq,
                               h.hkv, h.hd, max_ctx).cpu().numpy().astype(np.float64).reshape(q.shape)
    for s in range(B):
        want, bound = exact_rows(q[s].astype(np.float64), *h.history(s))
        assert np.all(np.abs(o[s] - want) <= bound), (s, np.max(np.abs(o[s] - want) / bound))


def one_component(h, hq):
    q = np.zeros((len(h.ctxs), hq, h.hd), dtype=np.float16)
    q[:, :, 0] = h.rng.uniform(0.7, 1.0, (len(h.ctxs), hq)) * math.sqrt(h.hd)
    return q


SHAPES = [(8, 8, 64), (8, 4, 128), (16, 4, 64), (32, 4, 128), (16, 2, 64), (4, 1, 128), (2, 1, 64), (2, 2, 128)]


@pytest.mark.parametrize("max_ctx", [100, 700])   # one CTA a pair; parts and their join
@pytest.mark.parametrize("hq,hkv,hd", SHAPES)
def test_probabilities_keep_their_bits(hq, hkv, hd, max_ctx):
    """Rows whose scores are exact, over values of one sign, so that what a probability loses shows."""
    h = EightBit(hq + hd + hkv, [33, 21, 100] if max_ctx == 100 else [33, 300, 700], hkv, hd, scale=-7, spread=1)
    h.codes[:, :, 1] &= 0x7F
    q = one_component(h, hq)
    check_exact(h, q, hq, max_ctx)


@pytest.mark.parametrize("max_ctx", [100, 700])
@pytest.mark.parametrize("hq,hkv,hd", SHAPES)
def test_small_values_beside_large_ones(hq, hkv, hd, max_ctx):
    """A token whose values are 2^15 times another's, in a component where the other's is 0: the
    others keep 2^-14 of theirs."""
    h = EightBit(hq + hd + hkv, [33, 40], hkv, hd, scale=-9, spread=0)
    h.codes[:, :, 1] &= 0x7F
    for s in range(2):
        b, slot = h.table[s, 0], 3 + s
        h.codes[b, :, 1, slot, 1:] = 0
        h.codes[b, :, 1, slot, 0] = int(np.searchsorted(GRID, 448.0))
        h.exps[b, :, 1, slot] = 6
    check_exact(h, one_component(h, hq), hq, max_ctx)
