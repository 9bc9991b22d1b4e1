"""Operators on the paged cache through the public entry points against the 64-bit
oracle: prompt attention, prompt weights, decode attention with weights,
eviction, and the four as a run of them is used."""
import math

import numpy as np
import pytest

import oracle
from tests.cache_cases import U32, History, prompt_reference, score_error

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import early_exit_decoding_layer_gb300 as ee  # noqa: E402

EE_DERR_LENGTH, EE_DERR_BLOCK = 16, 17


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from early_exit_decoding_layer_gb300 import build
    build.build()
    assert torch.cuda.is_available()


class Prompt:
    """Packed rows over a History: rows[s] new rows of sequence s, `lead` rows before
    the first sequence and `tail` behind the last that belong to none."""

    def __init__(self, seed, hq, hkv, hd, rows, ctxs, lead=0, tail=0):
        self.h = History(seed, ctxs, hkv, hd)
        self.hq, self.hkv, self.hd, self.rows = hq, hkv, hd, rows
        self.cu = np.concatenate([[lead], lead + np.cumsum(rows)]).astype(np.int32)
        self.T = int(self.cu[-1]) + tail
        self.q = self.h.rng.standard_normal((self.T, hq, hd)).astype(np.float16)
        self.q[:lead], self.q[self.cu[-1]:] = np.nan, np.nan
        self.max_ctx = max(max(ctxs), 1) + 5

    def args(self):
        d = {"q": dev(self.q.reshape(self.T, -1)), "k": dev(self.h.k), "v": dev(self.h.v), "table": dev(self.h.table),
             "cu": dev(self.cu), "ctx": dev(np.array(self.h.ctxs, dtype=np.int32))}
        return d

    @property
    def shape(self):
        return self.hq, self.hkv, self.hd, self.max_ctx

    def seq_rows(self, s):
        return slice(int(self.cu[s]), int(self.cu[s + 1]))


PROMPTS = [
    # one row, one token; a row tile's and a block's borders; several tiles
    (4, 2, 64, [1], [1]), (8, 8, 128, [16], [16]), (8, 1, 64, [17], [17]), (8, 2, 128, [129], [129]),
    (8, 8, 64, [255, 257], [255, 257]), (8, 4, 128, [300], [300]), (4, 2, 64, [640], [640]),
    # packs of odd lengths, some without rows, without tokens, or both
    (8, 2, 128, [3, 0, 130, 1], [3, 40, 130, 1]), (4, 2, 64, [0, 5, 0], [0, 5, 7]), (16, 2, 64, [33, 65, 31], [33, 65, 31]),
    # chunks behind a cached prefix: few rows, many tokens
    (8, 1, 128, [1, 7], [700, 33]), (4, 4, 64, [2], [1025]), (8, 2, 64, [60, 4], [400, 900]), (32, 8, 128, [1] * 3, [513, 16, 255]),
    # more rows than tokens: the first rows see nothing
    (8, 2, 64, [20, 9], [13, 0]), (4, 1, 128, [140], [12]),
]


@pytest.mark.parametrize("hq,hkv,hd,rows,ctxs", PROMPTS)
def test_prompt_attention_and_weights(hq, hkv, hd, rows, ctxs):
    c = Prompt(hq * 31 + hd + sum(rows), hq, hkv, hd, rows, ctxs, lead=2, tail=3)
    d = c.args()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((c.T, hq * hd), 7.0, dtype=torch.float16, device="cuda")
    o, lse = ee.prompt_attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["ctx"], *c.shape, out=out, err=err)
    w0 = np.where(c.h.owned()[:, None], 0.5, np.nan).astype(np.float32) * np.ones((1, hkv, 1), np.float32)
    w = dev(w0)
    lse0 = lse.clone()
    lse0[:, :2], lse0[:, int(c.cu[-1]):] = math.nan, math.nan   # rows of no sequence: not read
    ee.prompt_weights(d["q"], d["k"], d["table"], d["cu"], d["ctx"], lse0, w, *c.shape, err=err)
    assert err.item() == 0
    o, lse, w = o.cpu().numpy().astype(np.float64), lse.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    assert np.all(o[:2] == 7.0) and np.all(o[c.cu[-1]:] == 7.0)   # rows of no sequence: as they were
    o = o.reshape(c.T, hq, hd)
    for s in range(len(rows)):
        r = c.seq_rows(s)
        ro, rl, rw, bo, bl, bw = prompt_reference(c.h, s, c.q[r])
        assert np.all(np.abs(o[r] - ro) <= bo), (s, np.max(np.abs(o[r] - ro) - bo))
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(lse[:, r]), empty)
        assert np.all(np.abs(lse[:, r][~empty] - rl[~empty]) <= bl[~empty])
        got = c.h.gather(w, s)
        assert np.all(np.abs(got - 0.5 - rw) <= bw + U32 * (1 + rw)), (s, np.max(np.abs(got - 0.5 - rw) - bw))
    unowned = ~np.broadcast_to(c.h.owned()[:, None], w.shape)
    assert np.all(np.isnan(w[unowned]))


def test_prompt_strided_rows_and_repeat():
    """q and o as columns of wider rows; a second call gives the same bits."""
    c = Prompt(5, 8, 2, 64, [70, 33], [70, 90])
    d = c.args()
    wide = torch.full((c.T, 8 * 64 * 2 + 24), 3.0, dtype=torch.float16, device="cuda")
    wide[:, 8:8 + 512] = d["q"]
    q, out = wide[:, 8:8 + 512], wide[:, 520 + 8:520 + 8 + 512]
    ref, lse = ee.prompt_attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["ctx"], *c.shape)
    o, lse2 = ee.prompt_attention(q, d["k"], d["v"], d["table"], d["cu"], d["ctx"], *c.shape, out=out)
    assert torch.equal(o, ref) and torch.equal(lse, lse2)
    assert torch.all(wide[:, :8] == 3.0) and torch.all(wide[:, 520:528] == 3.0) and torch.all(wide[:, 1040:] == 3.0)
    ws = [torch.zeros(c.h.n_blocks, 2, 16, device="cuda") for _ in range(2)]
    for x, w in zip((d["q"], q), ws):
        ee.prompt_weights(x, d["k"], d["table"], d["cu"], d["ctx"], lse, w, *c.shape)
    assert torch.equal(*ws)


def test_prompt_nonfinite_tokens_reach_only_rows_that_see_them():
    """A NaN or infinite value belongs to its own token: rows before it do not see it."""
    hq, hkv, hd, n = 8, 2, 64, 200
    c = Prompt(11, hq, hkv, hd, [n], [n])
    d = c.args()
    clean, lse = ee.prompt_attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["ctx"], *c.shape)
    cells = {(70, 0, 5): np.nan, (133, 1, 40): np.inf, (199, 0, 63): -np.inf}
    v = c.h.v.copy()
    for (t, g, i), x in cells.items():
        v[c.h.table[0, t // 16], g, t % 16, i] = x
    o, lse2 = ee.prompt_attention(d["q"], d["k"], dev(v), d["table"], d["cu"], d["ctx"], *c.shape)
    want = clean.view(n, hq, hd).clone()
    for (t, g, i), x in cells.items():
        want[t:, g * 4:(g + 1) * 4, i] = x
    assert torch.equal(torch.nan_to_num(o.view(n, hq, hd), nan=777.0), torch.nan_to_num(want, nan=777.0))
    assert torch.equal(lse, lse2)
    # a NaN key makes every row that sees it NaN, and no other
    k = c.h.k.copy()
    k[c.h.table[0, 70 // 16], 1, 70 % 16, 3] = np.nan
    o, lse2 = ee.prompt_attention(d["q"], dev(k), d["v"], d["table"], d["cu"], d["ctx"], *c.shape)
    o = o.view(n, hq, hd)
    assert torch.equal(o[:70], clean.view(n, hq, hd)[:70]) and torch.equal(o[:, :4], clean.view(n, hq, hd)[:, :4])
    assert torch.isnan(o[70:, 4:]).all() and torch.isnan(lse2[4:, 70:]).all()


def test_prompt_sharp_rows():
    """Scores that differ by hundreds, growing and falling along the keys: the running
    maximum moves, and only the tokens near it count."""
    hq, hkv, hd, n = 4, 1, 64, 330
    c = Prompt(13, hq, hkv, hd, [n], [n])
    c.q[:] = 0
    c.q[:, :, 0] = [[8.0, -8.0, 1.0, 0.0]]
    ramp = (np.arange(n) * 0.25).astype(np.float16)
    for t in range(n):
        c.h.K[0][t] = 0
        c.h.K[0][t, 0, 0] = ramp[t]
        c.h.k[c.h.table[0, t // 16], 0, t % 16] = c.h.K[0][t, 0]
    d = c.args()
    o, lse = ee.prompt_attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["ctx"], *c.shape)
    ro, rl, _, bo, bl, _ = prompt_reference(c.h, 0, c.q)
    assert np.all(np.abs(o.cpu().numpy().astype(np.float64).reshape(n, hq, hd) - ro) <= bo)
    assert np.all(np.abs(lse.cpu().numpy() - rl) <= bl)


DECODE = [
    (4, 2, 64, [1]), (4, 2, 64, [0, 15, 16, 17]), (32, 8, 64, [300, 1, 47]), (32, 8, 128, [2304]), (64, 8, 128, [1100, 33]),
    (8, 8, 128, [5, 64, 129, 1000]), (16, 16, 64, [700, 0]), (8, 4, 128, [513, 31]), (4, 1, 64, [5000]),
]


def check_attention_weights(h, q, ctxs, hkv, table, max_ctx):
    """One call on history h against the formulas in 64 bits."""
    B, hq, hd = q.shape
    pos = dev(np.array(ctxs, dtype=np.int32) - 1)
    w, err = dev(h.w), torch.zeros(1, dtype=torch.int32, device="cuda")
    o = ee.attention_weights(dev(q.reshape(B, -1)), dev(h.k), dev(h.v), dev(table), pos, w, hq, hkv, hd, max_ctx, err=err)
    o, w = o.cpu().numpy().reshape(B, hq, hd), w.cpu().numpy()
    assert err.item() == 0
    g = np.arange(hq) * hkv // hq
    for s, c in enumerate(ctxs):
        if c == 0:
            assert np.all(o[s] == 0)
            continue
        K, V, q64 = h.K[s].astype(np.float64), h.V[s].astype(np.float64), q[s].astype(np.float64)
        ro, _, rw = oracle.prompt_attention(q64[None], K, V)
        z = np.einsum("hd,thd->th", q64, K[:, g]) / math.sqrt(hd)
        # scores, exp, sums of c terms, the division: as for a prompt, all in fp32
        rel = 2 * score_error(q64, K) + (c + 32) * U32 + 4 * U32 * np.abs(z).max(0)
        p = np.exp(z - z.max(0))
        p /= p.sum(0)
        bound = rel[:, None] * np.einsum("th,thd->hd", p, np.abs(V[:, g])) + 1e-30
        assert np.all(np.abs(o[s] - ro[0]) <= bound), s
        bw = np.zeros_like(rw)
        for a in range(hq):
            bw[:, g[a]] += p[:, a] * rel[a]
        got = h.gather(w, s)
        assert np.all(np.abs(got - h.W[s] - rw) <= bw + 8 * U32 * (h.W[s] + rw)), s
    unowned = ~np.broadcast_to(h.owned()[:, None], w.shape)
    assert np.all(np.isnan(w[unowned]))


@pytest.mark.parametrize("hq,hkv,hd,ctxs", DECODE)
def test_attention_weights(hq, hkv, hd, ctxs):
    h = History(hq + hd + sum(ctxs), ctxs, hkv, hd)
    q = h.rng.standard_normal((len(ctxs), hq, hd)).astype(np.float32)
    check_attention_weights(h, q, ctxs, hkv, h.table, max(ctxs) + 9)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("hq,hkv,hd,seqs", [(32, 8, 128, 40), (64, 8, 128, 20), (16, 16, 64, 33), (8, 4, 64, 64)])
def test_attention_weights_many_units(hq, hkv, hd, seqs, wide):
    """More (sequence, kv head) pairs than the GPU has SMs, so that every cluster has several
    one after another.  wide: room for 16384 tokens, of which few exist, so that clusters
    are large and some of their CTAs have nothing to do."""
    r = np.random.default_rng(seqs + hd)
    ctxs = [0, 1, 700] + [int(x) for x in np.exp(r.uniform(0, np.log(500), seqs - 3))]
    h = History(hq + seqs, ctxs, hkv, hd)
    q = h.rng.standard_normal((seqs, hq, hd)).astype(np.float32)
    table = np.full((seqs, 1024), 0x7FFFFFF0, dtype=np.int32)
    table[:, : h.table.shape[1]] = h.table
    check_attention_weights(h, q, ctxs, hkv, table, 16384 if wide else max(ctxs))


def test_attention_weights_agrees_with_attention():
    h = History(3, [777, 40], 8, 128)
    q = dev(h.rng.standard_normal((2, 32 * 128)).astype(np.float32))
    pos = dev(np.array([776, 39], dtype=np.int32))
    table = np.where(h.table == 0x7FFFFFF0, 0, h.table)
    kc, vc = dev(np.nan_to_num(h.k)), dev(np.nan_to_num(h.v))
    a = ee.attention(q, kc, vc, dev(table), pos, 32, 8, 128, 800)
    b = ee.attention_weights(q, kc, vc, dev(table), pos, dev(h.w), 32, 8, 128, 800)
    assert torch.allclose(a, b, rtol=1e-4, atol=1e-5)


EVICT = [
    (1, 64, [1], 1, 0), (2, 64, [40], 24, 5), (2, 128, [17, 16, 300, 0], 16, 16), (3, 64, [100, 65], 64, 0),
    (8, 128, [513, 90], 100, 7), (1, 128, [2000], 1999, 3), (2, 64, [1500, 700], 1, 1), (2, 64, [129], 128, 1),
    (1, 64, [5000], 2500, 100), (2, 64, [40, 7], 100, 50), (1, 128, [1], 16384, 16384),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("hkv,hd,ctxs,keep,recent", EVICT)
def test_evict(hkv, hd, ctxs, keep, recent, in_place):
    nd = (min(keep, max(ctxs) + 3) + 15) // 16
    h = History(hd + keep + sum(ctxs), ctxs, hkv, hd, spare=3 + len(ctxs) * nd)
    free = np.setdiff1d(np.arange(h.n_blocks), h.table)
    dst = h.table if in_place else h.rng.permutation(free)[: len(ctxs) * nd].astype(np.int32).reshape(len(ctxs), nd)
    k, v, w = dev(h.k), dev(h.v), dev(h.w)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, new = ee.evict(k, v, w, dev(h.table), dev(np.array(ctxs, dtype=np.int32)), keep, recent, max(ctxs) + 3,
                         dst_table=None if in_place else dev(dst), err=err)
    assert err.item() == 0
    kept, new, k, v, w = (x.cpu().numpy() for x in (kept, new, k, v, w))
    assert np.array_equal(new, np.minimum(ctxs, keep))
    touched = np.zeros((h.n_blocks, 16), dtype=bool)
    for s, c in enumerate(ctxs):
        n = min(c, keep)
        want = oracle.evict_indices(h.W[s], keep, recent)
        assert np.array_equal(kept[s, :, :n], want) and np.all(kept[s, :, n:] == -1)
        t = np.arange(n)
        touched[dst[s, t // 16], t % 16] = True
        for got, src in ((k, h.K[s]), (v, h.V[s]), (w, h.W[s])):
            moved = h.gather(got, s, n, dst)
            for g in range(hkv):
                assert np.array_equal(moved[:, g], src[want[g], g])
    for got, before in ((k, h.k), (v, h.v), (w, h.w)):   # all other slots as they were
        a, b = np.moveaxis(got, 2, 1)[~touched], np.moveaxis(before, 2, 1)[~touched]
        assert np.array_equal(a, b, equal_nan=True)


def test_evict_odd_weights():
    """NaN is lightest, -0 is 0, infinities and negative weights keep their order."""
    h = History(9, [48], 1, 64)
    w = np.full(48, 1.0, dtype=np.float32)
    w[[0, 5]], w[7], w[9], w[11], w[13], w[20:30] = np.nan, np.inf, -np.inf, -2.0, -0.0, 0.0
    w[31:40] = np.float32(1e-42)   # subnormal
    h.W[0][:, 0] = w
    for t in range(48):
        h.w[h.table[0, t // 16], 0, t % 16] = w[t]
    for keep in (47, 46, 45, 44, 43, 40, 35, 30, 20, 3, 1):
        kept, _ = ee.evict(dev(h.k), dev(h.v), dev(h.w), dev(h.table), dev(np.array([48], np.int32)), keep, 1, 48)
        assert np.array_equal(kept.cpu().numpy()[0], oracle.evict_indices(h.W[0], keep, 1)), keep


def test_prompt_decode_evict_run():
    """The four as they are used: a packed prompt, what its tokens weigh, two decode
    steps, an eviction in place, and a decode step over the smaller cache."""
    hq, hkv, hd, keep, recent = 8, 2, 128, 40, 8
    rows = [150, 61]
    h = History(21, [n + 3 for n in rows], hkv, hd)
    q = h.rng.standard_normal((sum(rows), hq, hd)).astype(np.float16)
    steps = h.rng.standard_normal((3, 2, hq, hd)).astype(np.float32)
    k, v, table = dev(h.k), dev(h.v), dev(h.table)
    w = torch.zeros(h.n_blocks, hkv, 16, device="cuda")
    shape = (hq, hkv, hd, 160)
    cu, n = dev(np.array([0, 150, 211], np.int32)), dev(np.array(rows, np.int32))
    qd = dev(q.reshape(-1, hq * hd))
    o, lse = ee.prompt_attention(qd, k, v, table, cu, n, *shape)
    ee.prompt_weights(qd, k, table, cu, n, lse, w, *shape)
    outs = [ee.attention_weights(dev(steps[i].reshape(2, -1)), k, v, table, n + i, w, *shape) for i in range(2)]
    kept, new = ee.evict(k, v, w, table, n + 2, keep, recent, 160)
    outs.append(ee.attention_weights(dev(steps[2].reshape(2, -1)), k, v, table, new - 1, w, *shape))
    assert new.tolist() == [keep, keep]
    kept, w = kept.cpu().numpy(), w.cpu().numpy()
    for s, r in enumerate(rows):
        K, V = h.K[s].astype(np.float64), h.V[s].astype(np.float64)
        rows_q = q[sum(rows[:s]):sum(rows[:s + 1])]
        ro, _, weight, bo, _, bw = prompt_reference(h, s, rows_q, ctx=r)
        got = o.cpu().numpy().astype(np.float64).reshape(-1, hq, hd)[sum(rows[:s]):sum(rows[:s + 1])]
        assert np.all(np.abs(got - ro) <= bo)
        total, bound = np.zeros((r + 2, hkv)), np.zeros((r + 2, hkv))
        total[:r], bound[:r] = weight, bw
        for i in range(2):
            c = r + i + 1
            x, _, p = oracle.prompt_attention(steps[i, s][None].astype(np.float64), K[:c], V[:c])
            assert np.allclose(outs[i].cpu().numpy()[s].reshape(hq, hd), x[0], rtol=1e-4, atol=1e-5)
            total[:c] += p
        bound += 1e-4 * total + 1e-6   # the decode steps' tolerance, as for attention()
        for g in range(hkv):
            ks = kept[s, g]
            assert np.all(np.diff(ks) > 0) and np.array_equal(ks[-recent:], np.arange(r + 2 - recent, r + 2))
            left = np.setdiff1d(np.arange(r + 2), ks)
            heavy = ks[:-recent]
            assert np.all(total[heavy, g, None] + bound[heavy, g, None] >= total[left, g] - bound[left, g])
            # the next step sees the kept tokens alone
            x, _, p = oracle.prompt_attention(steps[2, s][None, g * 4:(g + 1) * 4].astype(np.float64), K[ks][:, g:g + 1],
                                              V[ks][:, g:g + 1])
            y = outs[2].cpu().numpy()[s].reshape(hq, hd)[g * 4:(g + 1) * 4]
            assert np.allclose(y, x[0], rtol=1e-4, atol=1e-5)
            assert np.allclose(h.gather(w, s, keep)[:, g], total[ks, g] + p[:, 0], rtol=2e-4, atol=1e-5)


def test_shared_prefix_blocks():
    """Two sequences over the same first blocks: read as each one's own, weights get both
    parts."""
    h = History(31, [64, 50], 2, 64)
    h.table[1, :2] = h.table[0, :2]
    for x in (h.K, h.V):
        x[1][:32] = x[0][:32]
    q = h.rng.standard_normal((82, 4, 64)).astype(np.float16)
    cu, ctx = dev(np.array([0, 64, 82], np.int32)), dev(np.array([64, 50], np.int32))
    w = torch.zeros(h.n_blocks, 2, 16, device="cuda")
    o, lse = ee.prompt_attention(dev(q.reshape(82, -1)), dev(h.k), dev(h.v), dev(h.table), cu, ctx, 4, 2, 64, 64)
    ee.prompt_weights(dev(q.reshape(82, -1)), dev(h.k), dev(h.table), cu, ctx, lse, w, 4, 2, 64, 64)
    refs = [prompt_reference(h, s, q[[0, 64][s]:[64, 82][s]]) for s in range(2)]
    o, w = o.cpu().numpy().astype(np.float64).reshape(82, 4, 64), w.cpu().numpy()
    for s in range(2):
        assert np.all(np.abs(o[[0, 64][s]:[64, 82][s]] - refs[s][0]) <= refs[s][3])
    both, bound = refs[0][2].copy(), refs[0][5].copy()
    both[:32] += refs[1][2][:32]
    bound[:32] += refs[1][5][:32]
    assert np.all(np.abs(h.gather(w, 0) - both) <= bound + 4 * U32 * both)


def test_capture_replay_and_streams():
    """A captured run replays on new inputs; another captured run of the same operators
    on another stream shares nothing with it."""
    runs = []
    for i in range(2):
        c = Prompt(41 + i, 8, 2, 64, [90, 20], [90, 300])
        d = c.args()
        d["w"] = torch.zeros(c.h.n_blocks, 2, 16, device="cuda")
        d["out"] = torch.zeros(c.T, 512, dtype=torch.float16, device="cuda")
        d["qd"] = dev(c.h.rng.standard_normal((2, 512)).astype(np.float32))
        d["dst"] = d["table"]

        def run(c=c, d=d):
            o, lse = ee.prompt_attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["ctx"], *c.shape, out=d["out"])
            ee.prompt_weights(d["q"], d["k"], d["table"], d["cu"], d["ctx"], lse, d["w"], *c.shape)
            x = ee.attention_weights(d["qd"], d["k"], d["v"], d["table"], d["ctx"] - 1, d["w"], *c.shape)
            kept, new = ee.evict(d["k"], d["v"], d["w"], d["table"], d["ctx"], 50, 10, c.max_ctx)
            return o, lse, x, kept, new

        fresh = {n: t.clone() for n, t in d.items()}
        eager = [t.clone() for t in run()] + [d[n].clone() for n in ("k", "v", "w")]

        def restore(d=d, fresh=fresh):
            for n, t in fresh.items():
                d[n].copy_(t)

        restore()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            run()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=stream):
                outs = run()
            restore()
        runs.append((graph, stream, outs, eager, d, restore))
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream, *_rest in runs:
            _rest[-1]()
        torch.cuda.synchronize()
        for graph, stream, *_rest in runs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for graph, stream, outs, eager, d, _ in runs:
            for a, b in zip(list(outs) + [d[n] for n in ("k", "v", "w")], eager):
                assert torch.equal(torch.nan_to_num(a.float(), nan=777.0), torch.nan_to_num(b.float(), nan=777.0))


def test_bad_lengths_and_blocks_are_reported():
    """The kernels' own checks: the call stays inside the arrays and the error word
    says what was wrong; sequences without a fault are right."""
    c = Prompt(51, 4, 2, 64, [20, 30], [20, 30])
    d = c.args()
    good, _ = ee.prompt_attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["ctx"], *c.shape)

    def calls(table, ctx, cu, err):
        w = torch.zeros(c.h.n_blocks, 2, 16, device="cuda")
        k, v = d["k"].clone(), d["v"].clone()
        o, lse = ee.prompt_attention(d["q"], k, v, table, cu, ctx, *c.shape, err=err[0])
        ee.prompt_weights(d["q"], k, table, cu, ctx, lse, w, *c.shape, err=err[1])
        ee.attention_weights(d["q"][:2].float(), k, v, table, ctx - 1, w, *c.shape, err=err[2])
        ee.evict(k, v, w, table, ctx, 7, 2, c.max_ctx, err=err[3])
        return o

    for what, code in (("block", EE_DERR_BLOCK), ("negative block", EE_DERR_BLOCK), ("long", EE_DERR_LENGTH),
                       ("negative", EE_DERR_LENGTH)):
        table, ctx = d["table"].clone(), d["ctx"].clone()
        if "block" in what:
            table[0, 1] = -3 if "negative" in what else c.h.n_blocks
        else:
            ctx[0] = -5 if what == "negative" else 1 << 30
            table[0] = table[1]   # whatever is read lies in the cache
            table[0, 2:] = 0
        err = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(4)]
        o = calls(table, ctx, d["cu"], err)
        assert [e.item() for e in err] == [code] * 4, what
        assert torch.equal(o[20:], good[20:]), what
    err = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(4)]
    calls(d["table"], d["ctx"], dev(np.array([0, 20, 1 << 30], np.int32)), err)
    assert [e.item() for e in err[:2]] == [EE_DERR_LENGTH] * 2


def test_refusals_on_device_tensors():
    c = Prompt(61, 4, 2, 64, [20], [20])
    d = c.args()
    w = torch.zeros(c.h.n_blocks, 2, 16, device="cuda")
    ok = dict(q=d["q"], k=d["k"], v=d["v"], table=d["table"], cu=d["cu"], ctx=d["ctx"])

    def attn(shape=c.shape, **kw):
        a = {**ok, **kw}
        return ee.prompt_attention(a["q"], a["k"], a["v"], a["table"], a["cu"], a["ctx"], *shape, out=a.get("out"))

    attn()
    bad = [dict(q=d["q"].float()), dict(q=d["q"].cpu()), dict(k=d["k"][:, :, :, :32]), dict(v=d["v"][1:]),
           dict(table=d["table"].long()), dict(cu=d["cu"][:1]), dict(ctx=d["ctx"].cpu()), dict(out=d["q"]),
           dict(out=torch.zeros(19, 256, dtype=torch.float16, device="cuda")), dict(q=d["q"].t().contiguous().t()),
           dict(shape=(4, 2, 64, 0)), dict(shape=(4, 2, 64, 16385)), dict(shape=(6, 2, 64, 25))]
    for kw in bad:
        with pytest.raises(ee.EEError) as e:
            attn(**kw)
        assert e.value.status == 1, kw
    for kw in (dict(keep=0), dict(recent=-1), dict(recent=9), dict(keep=16385), dict(dst_table=d["table"][:, :0])):
        with pytest.raises(ee.EEError) as e:
            ee.evict(d["k"], d["v"], w, d["table"], d["ctx"], **{"keep": 8, "recent": 2, "max_ctx": 20, **kw})
        assert e.value.status == 1, kw
    for kw, error in ((dict(keep=1 << 40), ee.EEError), (dict(max_ctx=-(1 << 70)), ee.EEError), (dict(recent=2.5), TypeError),
                      (dict(err=w), ee.EEError)):
        with pytest.raises(error):
            ee.evict(d["k"], d["v"], w, d["table"], d["ctx"], **{"keep": 8, "recent": 2, "max_ctx": 20, **kw})
    with pytest.raises(ee.EEError):
        ee.attention_weights(d["q"][:1], d["k"], d["v"], d["table"], d["ctx"], w, *c.shape)   # fp16 queries
    with pytest.raises(ee.EEError):
        ee.prompt_weights(d["q"], d["k"], d["table"], d["cu"], d["ctx"], torch.zeros(4, 19, device="cuda"), w, *c.shape)
    torch.cuda.synchronize()


def far_caches(h, shift):
    """h's caches with every block `shift` ids further on, in arrays whose elements before
    are left as the allocator gave them."""
    out = []
    for a in (h.k, h.v, h.w):
        x = torch.empty((shift + h.n_blocks,) + a.shape[1:], dtype=torch.from_numpy(a).dtype, device="cuda")
        x[shift:] = dev(a)
        out.append(x)
    return out + [dev(np.where(h.table == 0x7FFFFFF0, h.table, h.table + shift))]


def test_offsets_beyond_32_bits():
    """Blocks whose elements lie behind 2^32 bytes and 2^31 elements: the same bits as
    near the start."""
    hq, hkv, hd = 32, 8, 128
    c = Prompt(71, hq, hkv, hd, [70, 9], [70, 200])
    shift = (1 << 31) // (hkv * 16 * hd) + 1000
    near = [dev(c.h.k), dev(c.h.v), dev(c.h.w), dev(c.h.table)]
    far = far_caches(c.h, shift)
    d = c.args()
    qd = dev(c.h.rng.standard_normal((2, hq * hd)).astype(np.float32))
    got = []
    for k, v, w, table in (near, far):
        o, lse = ee.prompt_attention(d["q"], k, v, table, d["cu"], d["ctx"], *c.shape)
        ee.prompt_weights(d["q"], k, table, d["cu"], d["ctx"], lse, w, *c.shape)
        x = ee.attention_weights(qd, k, v, table, d["ctx"] - 1, w, *c.shape)
        kept, new = ee.evict(k, v, w, table, d["ctx"], 33, 5, c.max_ctx)
        n = c.h.n_blocks
        got.append([o, lse, x, kept, new, k[-n:].clone(), v[-n:].clone(), w[-n:].clone()])
    for a, b in zip(*got):
        assert torch.equal(torch.nan_to_num(a.float(), nan=777.0), torch.nan_to_num(b.float(), nan=777.0))


@pytest.mark.parametrize("hq,hkv,hd", [(8, 2, 128), (8, 1, 64)])
def test_longest_prompt(hq, hkv, hd):
    """16384 tokens: rows from all over against 64 bits, every row's weights adding up to
    one, the last row as a decode step, and the eviction to half."""
    n, T = 16384, torch.float64
    g = torch.Generator(device="cuda").manual_seed(5)
    nb = n // 16
    k, v = (torch.randn(nb, hkv, 16, hd, generator=g, device="cuda").half() for _ in range(2))
    table = torch.randperm(nb, generator=g, device="cuda").to(torch.int32).view(1, nb)
    q = torch.randn(n, hq * hd, generator=g, device="cuda").half()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    w = torch.zeros(nb, hkv, 16, device="cuda")
    shape = (hq, hkv, hd, n)
    o, lse = ee.prompt_attention(q, k, v, table, i32(0, n), i32(n), *shape)
    ee.prompt_weights(q, k, table, i32(0, n), i32(n), lse, w, *shape)
    flat = lambda x: x[table[0].long()].transpose(1, 2).reshape(n, hkv, -1)  # noqa: E731
    K, V, W = flat(k).to(T), flat(v).to(T), flat(w)[..., 0]
    G = hq // hkv
    for r in (0, 1, 63, 64, 127, 128, 255, 4095, 8191, 16320, 16383):
        z = torch.einsum("hgd,thd->hgt", q[r].view(hkv, G, hd).to(T), K[: r + 1]) / math.sqrt(hd)
        p = torch.softmax(z, -1)
        ref = torch.einsum("hgt,thd->hgd", p, V[: r + 1])
        mag = torch.einsum("hgt,thd->hgd", p, V[: r + 1].abs())
        # as in prompt_reference: fp16 probabilities (2^-11 relative, 2^-25 absolute) and result
        bound = (2.0 ** -11 + 1e-4) * mag + 2.0 ** -25 * V[: r + 1].abs().sum(0)[:, None] + 2.0 ** -11 * ref.abs() * 1.001 + 2.0 ** -25
        assert torch.all((o[r].view(hkv, G, hd).to(T) - ref).abs() <= bound), r
        # sums of r + 1 terms in fp32 and a score's error, as in prompt_reference
        assert torch.all((lse[:, r].view(hkv, G).to(T) - torch.logsumexp(z, -1)).abs() <= 1e-4), r
    # every row gives one weight per head of the group: n G per kv head, each to 2e-5
    assert torch.all((W.to(T).sum(0) - n * G).abs() <= 2e-5 * n * G)
    # the last tokens' weights come from few rows
    rows = slice(n - 40, n)
    z = torch.einsum("rhgd,thd->hgrt", q[rows].view(40, hkv, G, hd).to(T), K) / math.sqrt(hd)
    seen = torch.arange(n, device="cuda") <= torch.arange(n - 40, n, device="cuda")[:, None]
    p = torch.softmax(z.masked_fill(~seen, -math.inf), -1).sum((1, 2))
    assert torch.allclose(W[n - 40:].T.to(T), p[:, n - 40:], rtol=1e-4, atol=0)
    # decode: the same row from fp32 queries
    before = w.clone()
    x = ee.attention_weights(q[-1:].float(), k, v, table, i32(n - 1), w, *shape)
    assert torch.all((x[0].view(hkv, G, hd).to(T) - ref).abs() <= 1e-4 * mag)
    add = (flat(w)[..., 0] - flat(before)[..., 0]).to(T)
    assert torch.all((add.sum(0) - G).abs() <= 1e-2)   # added to sums of up to 10^4, rounded there
    # eviction: ties at the border go to the lower index
    flat_w = torch.round(flat(w)[..., 0] * 4) / 4
    wq = torch.empty_like(w)
    wq[table[0].long()] = flat_w.view(nb, 16, hkv).transpose(1, 2)
    kept, new = ee.evict(k, v, wq, table, i32(n), n // 2, 100, n)
    want = oracle.evict_indices(flat_w.cpu().numpy(), n // 2, 100)
    assert new.item() == n // 2 and np.array_equal(kept[0].cpu().numpy(), want)
    moved = flat(k)[: n // 2].cpu()
    for h in range(hkv):
        assert torch.equal(moved[:, h], K[want[h], h].half().cpu())


def test_full_batch():
    """64 sequences, some without rows or tokens: every operator, each sequence as its own."""
    hq, hkv, hd = 8, 2, 64
    rng = np.random.default_rng(81)
    ctxs = [int(x) for x in rng.integers(0, 90, 64)]
    ctxs[3] = ctxs[63] = 0
    rows = [int(min(c, x)) for c, x in zip(ctxs, rng.integers(0, 60, 64))]
    c = Prompt(82, hq, hkv, hd, rows, ctxs, lead=1, tail=1)
    d = c.args()
    w = torch.zeros(c.h.n_blocks, hkv, 16, device="cuda")
    o, lse = ee.prompt_attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["ctx"], *c.shape)
    ee.prompt_weights(d["q"], d["k"], d["table"], d["cu"], d["ctx"], lse, w, *c.shape)
    qd = c.h.rng.standard_normal((64, hq, hd)).astype(np.float32)
    x = ee.attention_weights(dev(qd.reshape(64, -1)), d["k"], d["v"], d["table"], d["ctx"] - 1, w, *c.shape)
    kept, new = ee.evict(d["k"], d["v"], dev(c.h.w), d["table"], d["ctx"], 20, 4, c.max_ctx)
    o, lse, x, w, kept, new = (t.cpu().numpy() for t in (o, lse, x, w, kept, new))
    o = o.astype(np.float64).reshape(c.T, hq, hd)
    for s in range(64):
        r = c.seq_rows(s)
        ro, rl, rw, bo, bl, bw = prompt_reference(c.h, s, c.q[r])
        assert np.all(np.abs(o[r] - ro) <= bo) and np.all(np.abs(lse[:, r] - rl) <= bl), s
        n = min(ctxs[s], 20)
        assert new[s] == n
        if ctxs[s] == 0:
            assert np.all(x[s] == 0)
            continue
        xo, _, p = oracle.prompt_attention(qd[s][None].astype(np.float64), c.h.K[s].astype(np.float64), c.h.V[s].astype(np.float64))
        assert np.allclose(x[s].reshape(hq, hd), xo[0], rtol=1e-4, atol=1e-5), s
        assert np.all(np.abs(c.h.gather(w, s) - rw - p) <= bw + 1e-4 * (rw + p) + 1e-6), s
        assert np.array_equal(kept[s, :, :n], oracle.evict_indices(c.h.W[s], 20, 4)), s


@pytest.mark.parametrize("hq,hkv,hd,most", [(32, 32, 64, 100), (64, 16, 128, 31), (16, 16, 128, 140)])
def test_many_small_units(hq, hkv, hd, most):
    """More (row tile, kv head) pairs than SMs, most of them with one row tile of two, some
    whose first rows see nothing: every CTA goes through several of them."""
    rng = np.random.default_rng(hq + hd)
    rows = [int(x) for x in rng.integers(1, most, 64)]
    rows[::7] = [2 * most] * len(rows[::7])
    ctxs = [max(0, r + int(x)) for r, x in zip(rows, rng.integers(-most // 2, 40, 64))]
    c = Prompt(91, hq, hkv, hd, rows, ctxs)
    d = c.args()
    w = torch.zeros(c.h.n_blocks, hkv, 16, device="cuda")
    first = None
    for _ in range(3):
        o, lse = ee.prompt_attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["ctx"], *c.shape)
        first = (o, lse) if first is None else first
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    ee.prompt_weights(d["q"], d["k"], d["table"], d["cu"], d["ctx"], lse, w, *c.shape)
    o, lse, w = (t.cpu().numpy() for t in (o, lse, w))
    o = o.astype(np.float64).reshape(c.T, hq, hd)
    G = hq // hkv
    for s in range(0, 64, 5):
        r = c.seq_rows(s)
        for g in (0, hkv // 2, hkv - 1):   # a kv head's group at a time: the oracle's loops stay short
            one = History.__new__(History)
            one.K, one.V = [c.h.K[s][:, g:g + 1]], [c.h.V[s][:, g:g + 1]]
            heads = slice(g * G, (g + 1) * G)
            ro, rl, rw, bo, bl, bw = prompt_reference(one, 0, c.q[r][:, heads])
            assert np.all(np.abs(o[r, heads] - ro) <= bo), (s, g)
            got, seen = lse[heads, r], ~np.isneginf(rl)
            assert np.array_equal(~np.isneginf(got), seen) and np.all(np.abs(got[seen] - rl[seen]) <= bl[seen]), (s, g)
            assert np.all(np.abs(c.h.gather(w, s)[:, g] - rw[:, 0]) <= bw[:, 0] + U32 * rw[:, 0]), (s, g)


def test_first_call_may_be_captured():
    """The first call of each operator in a process, made while a stream is captured."""
    import subprocess
    import sys
    from tests.conftest import ROOT
    code = """
import torch
import early_exit_decoding_layer_gb300 as ee
d = "cuda"
q = torch.randn(20, 256, device=d).half()
k, v = (torch.randn(4, 2, 16, 64, device=d).half() for _ in range(2))
w = torch.zeros(4, 2, 16, device=d)
t = torch.arange(4, dtype=torch.int32, device=d).view(1, 4)
cu, n = torch.tensor([0, 20], dtype=torch.int32, device=d), torch.tensor([20], dtype=torch.int32, device=d)
q1, pos = q[-1:].float().contiguous(), n - 1
torch.cuda.synchronize()
g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(g, stream=s):
    o, lse = ee.prompt_attention(q, k, v, t, cu, n, 4, 2, 64, 64)
    ee.prompt_weights(q, k, t, cu, n, lse, w, 4, 2, 64, 64)
    x = ee.attention_weights(q1, k, v, t, pos, w, 4, 2, 64, 64)
    kept, new = ee.evict(k, v, w, t, n, 8, 2, 64)
g.replay()
torch.cuda.synchronize()
assert new.item() == 8 and torch.allclose(x[0], o[-1].float(), atol=5e-3), (x[0] - o[-1].float()).abs().max()
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ok" in r.stdout, r.stderr[-2000:]
