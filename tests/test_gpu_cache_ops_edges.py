"""The operators on the paged cache where they are easy to get wrong: CTAs without work
among others, values that are not finite, scores of extreme size, faulty lengths and
block ids next to sequences without a fault."""
import math

import numpy as np
import pytest

import oracle
from tests.cache_cases import U32, History, score_error
from tests.test_gpu_cache_ops import EE_DERR_BLOCK, EE_DERR_LENGTH, Prompt, check_attention_weights, dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import early_exit_decoding_layer_gb300 as ee  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from early_exit_decoding_layer_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("hq,hkv,hd", [(32, 8, 128), (16, 16, 64), (64, 8, 64)])
def test_attention_weights_ranks_without_tiles(hq, hkv, hd):
    """Room for 16384 tokens makes clusters large: 13 blocks leave some of their CTAs
    without a tile, 12 or 11 blocks give them one again, and sequences of a block or none
    leave nearly all of them without for many units in a row."""
    ctxs = [208, 192, 201, 177, 207, 190] * 3 + [1, 2, 0, 16] * 11 + [97, 0]
    h = History(hq + hd, ctxs, hkv, hd)
    q = h.rng.standard_normal((len(ctxs), hq, hd)).astype(np.float32)
    table = np.full((len(ctxs), 1024), 0x7FFFFFF0, dtype=np.int32)
    table[:, : h.table.shape[1]] = h.table
    check_attention_weights(h, q, ctxs, hkv, table, 16384)
    # again and again: the same bits, and no wait that ran out
    args = [dev(x) for x in (q.reshape(len(ctxs), -1), h.k, h.v, table, np.array(ctxs, dtype=np.int32) - 1)]
    err, first = torch.zeros(1, dtype=torch.int32, device="cuda"), None
    for _ in range(20):
        w = torch.zeros(h.n_blocks, hkv, 16, device="cuda")
        o = ee.attention_weights(*args, w, hq, hkv, hd, 16384, err=err)
        first = (o, w) if first is None else first
        assert torch.equal(o, first[0]) and torch.equal(w, first[1])
    assert err.item() == 0


# ------------------------------------------------ values that are not finite

def sharpen(h, s, q, t0):
    """Scores of sequence s's tokens from t0 on about 256 above those before, whatever the
    row: exp of the difference is 0 in fp32."""
    q[..., 0] = 16.0
    step = np.float16(16.0 * math.sqrt(h.hd))
    for t in range(h.ctxs[s]):
        h.K[s][t, :, 0] = step if t >= t0 else 0
        h.k[h.table[s, t // 16], :, t % 16, 0] = h.K[s][t, :, 0]


def bits(x):
    return torch.nan_to_num(x.float(), nan=777.0, posinf=888.0, neginf=999.0)


# keys of every unit split over six CTAs; over two; not split
SPLITS = [(8, 2, 64, [70], [2100]), (4, 1, 128, [9, 30], [640, 40]), (8, 8, 128, [300, 3] * 10, [300, 290] * 10)]


@pytest.mark.parametrize("sharp", [False, True])
@pytest.mark.parametrize("hq,hkv,hd,rows,ctxs", SPLITS)
def test_prompt_attention_nonfinite_visible_values(hq, hkv, hd, rows, ctxs, sharp):
    """A value that is not finite reaches every row that sees its token, in its own component
    alone, however small the token's probability and whichever CTA has it."""
    c = Prompt(hq + hd + sum(rows), hq, hkv, hd, rows, ctxs)
    n, ctx, G = rows[0], ctxs[0], hq // hkv
    if sharp:
        sharpen(c.h, 0, c.q[:n], ctx - n - 40 if ctx > n + 40 else ctx // 2)
    d = c.args()
    clean, lse = ee.prompt_attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["ctx"], *c.shape)
    # of an early tile, of the last tile before the rows' own, of a tile that some rows see in part
    cells = {(3, 0, 5): np.inf, (7, hkv - 1, 6): np.nan, (130, 0, 9): -np.inf, (ctx - n // 2, hkv - 1, 11): np.inf,
             (ctx - n, 0, 40): np.nan, (ctx - 1, 0, hd - 1): -np.inf}
    v = c.h.v.copy()
    hit = torch.zeros(c.T, hq, hd, dtype=torch.bool, device="cuda")
    for (t, g, i), x in cells.items():
        v[c.h.table[0, t // 16], g, t % 16, i] = x
        hit[max(0, t - (ctx - n)):n, g * G:(g + 1) * G, i] = True
    o, lse2 = ee.prompt_attention(d["q"], d["k"], dev(v), d["table"], d["cu"], d["ctx"], *c.shape)
    o, clean = o.view(c.T, hq, hd), clean.view(c.T, hq, hd)
    assert torch.isfinite(clean).all() and torch.equal(lse, lse2)
    assert not torch.isfinite(o[hit]).any()
    assert torch.equal(o[~hit], clean[~hit])


@pytest.mark.parametrize("sharp", [False, True])
@pytest.mark.parametrize("hq,hkv,hd,rows,ctxs", SPLITS)
def test_prompt_attention_nan_key(hq, hkv, hd, rows, ctxs, sharp):
    """A NaN key makes the rows that see it NaN, their log-sum-exp too, and no others."""
    c = Prompt(hq + hd + sum(rows), hq, hkv, hd, rows, ctxs)
    n, ctx, G = rows[0], ctxs[0], hq // hkv
    if sharp:
        sharpen(c.h, 0, c.q[:n], ctx - n - 40 if ctx > n + 40 else ctx // 2)
    d = c.args()
    clean, lse = ee.prompt_attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["ctx"], *c.shape)
    for t in (3, ctx - n // 2):
        k = c.h.k.copy()
        k[c.h.table[0, t // 16], hkv - 1, t % 16, 8] = np.nan
        hit = torch.zeros(c.T, hq, dtype=torch.bool, device="cuda")
        hit[max(0, t - (ctx - n)):n, (hkv - 1) * G:] = True
        o, lse2 = ee.prompt_attention(d["q"], dev(k), d["v"], d["table"], d["cu"], d["ctx"], *c.shape)
        o = o.view(c.T, hq, hd)
        assert torch.isnan(o[hit]).all() and torch.isnan(lse2.t()[hit]).all(), t
        assert torch.equal(o[~hit], clean.view(c.T, hq, hd)[~hit]) and torch.equal(lse2.t()[~hit], lse.t()[~hit]), t


# sequences on clusters, and more of them than SMs
DECODE = [(8, 2, 64, [2100]), (32, 8, 128, [2304, 700]), (4, 4, 128, [290, 600, 33] * 21)]


@pytest.mark.parametrize("sharp", [False, True])
@pytest.mark.parametrize("hq,hkv,hd,ctxs", DECODE)
def test_attention_weights_nonfinite(hq, hkv, hd, ctxs, sharp):
    """The same of decode steps: a value reaches its component of the group's heads, a NaN key
    all their outputs and the weight of every token of its kv head."""
    h = History(hq + hd + sum(ctxs), ctxs, hkv, hd)
    B, G, c = len(ctxs), hq // hkv, ctxs[0]
    q = h.rng.standard_normal((B, hq, hd)).astype(np.float32)
    if sharp:
        sharpen(h, 0, q[0], c - 20)
    pos, table = dev(np.array(ctxs, dtype=np.int32) - 1), dev(h.table)

    def call(k, v):
        w = dev(h.w)
        o = ee.attention_weights(dev(q.reshape(B, -1)), dev(k), dev(v), table, pos, w, hq, hkv, hd, max(ctxs))
        return o.view(B, hq, hd), w

    clean, w0 = call(h.k, h.v)
    assert torch.isfinite(clean).all()
    v, hit = h.v.copy(), torch.zeros(B, hq, hd, dtype=torch.bool, device="cuda")
    for (t, g, i), x in {(3, 0, 5): np.inf, (140, hkv - 1, 6): np.nan, (c - 1, 0, hd - 1): -np.inf, (c - 150, 0, 9): -np.inf}.items():
        v[h.table[0, t // 16], g, t % 16, i] = x
        hit[0, g * G:(g + 1) * G, i] = True
    o, w = call(h.k, v)
    assert not torch.isfinite(o[hit]).any()
    assert torch.equal(o[~hit], clean[~hit]) and torch.equal(bits(w), bits(w0))
    for t in (3, c - 150, c - 1):
        k, hit = h.k.copy(), torch.zeros(B, hq, dtype=torch.bool, device="cuda")
        k[h.table[0, t // 16], hkv - 1, t % 16, 8] = np.nan
        hit[0, (hkv - 1) * G:] = True
        o, w = call(k, h.v)
        assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], clean[~hit]), t
        own = np.zeros(h.w.shape, dtype=bool)
        own[h.table[0, np.arange(c) // 16], hkv - 1, np.arange(c) % 16] = True
        own = dev(own)
        assert torch.isnan(w[own]).all() and torch.equal(bits(w[~own]), bits(w0[~own])), t


def test_attention_weights_all_scores_minus_infinity():
    """A head whose scores are all -infinity weighs nothing: o = 0, as prompt_attention has it,
    and no weight is added; the other heads' are."""
    hq, hkv, hd, c = 4, 2, 64, 300
    h = History(17, [c, 40], hkv, hd)
    q = h.rng.standard_normal((2, hq, hd)).astype(np.float32)
    # sequence 0, kv head 0: keys of -infinity in dimension 0, the only one its two heads ask for
    q[0, :2] = 0
    q[0, :2, 0] = 1.0
    t = np.arange(c)
    k = h.k.copy()
    k[h.table[0, t // 16], 0, t % 16, 0] = -np.inf
    pos, table = dev(np.array([c - 1, 39], dtype=np.int32)), dev(h.table)
    out = []
    for kk in (h.k, k):
        w = dev(h.w)
        out.append((ee.attention_weights(dev(q.reshape(2, -1)), dev(kk), dev(h.v), table, pos, w, hq, hkv, hd, 320), w))
    (o0, w0), (o, w) = out
    o0, o = o0.view(2, hq, hd), o.view(2, hq, hd)
    assert torch.all(o[0, :2] == 0) and torch.equal(o[0, 2:], o0[0, 2:]) and torch.equal(o[1], o0[1])
    got, before = h.gather(w.cpu().numpy(), 0), h.W[0]
    assert np.array_equal(got[:, 0], before[:, 0])
    assert np.array_equal(got[:, 1], h.gather(w0.cpu().numpy(), 0)[:, 1])


@pytest.mark.parametrize("hq,hkv,hd,n,ctx", [(8, 2, 64, 200, 200), (8, 1, 128, 150, 420), (4, 4, 64, 700, 700), (16, 8, 64, 5, 90)])
def test_prompt_weights_of_rows_that_do_not_count(hq, hkv, hd, n, ctx):
    """A row's log-sum-exp of NaN reaches the tokens that the row sees and no others; a row
    whose log-sum-exp is -infinity adds nothing, whatever its queries are."""
    c = Prompt(hq + n, hq, hkv, hd, [n, 30], [ctx, 50])
    d, G, off = c.args(), hq // hkv, ctx - n
    _, lse = ee.prompt_attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["ctx"], *c.shape)

    def weights(q, lse):
        w = torch.zeros(c.h.n_blocks, hkv, 16, device="cuda")
        ee.prompt_weights(q, d["k"], d["table"], d["cu"], d["ctx"], lse, w, *c.shape)
        w = w.cpu().numpy()
        return c.h.gather(w, 0), c.h.gather(w, 1)

    clean, other = weights(d["q"], lse)
    q = d["q"].clone().view(c.T, hq, hd)
    for r in (n // 2, n - 1, 0):
        bad = lse.clone()
        bad[G - 1, r] = math.nan
        got, o = weights(d["q"], bad)
        assert np.isnan(got[: off + r + 1, 0]).all(), r
        assert np.array_equal(got[off + r + 1:, 0], clean[off + r + 1:, 0]), r
        assert np.array_equal(got[:, 1:], clean[:, 1:]) and np.array_equal(o, other), r
        off_row = lse.clone()
        off_row[:, r] = -math.inf
        want, _ = weights(d["q"], off_row)
        for x in (math.nan, math.inf, -math.inf):
            q2 = q.clone()
            q2[r, :, 3] = x
            got, o = weights(q2.view(c.T, -1), off_row)
            assert np.array_equal(got, want) and np.array_equal(o, other), (r, x)


@pytest.mark.parametrize("power", [-100, -70, 58, 70, 80, 110])
@pytest.mark.parametrize("hq,hkv,hd", [(8, 2, 64), (8, 8, 128)])
def test_attention_weights_queries_of_any_size(hq, hkv, hd, power):
    """Queries of 2^power: far down every token weighs the same, far up one has all the
    weight.  Scores are within fp32 in all of them."""
    ctxs = [300, 45]
    h = History(power + 200 + hd, ctxs, hkv, hd)
    q = (h.rng.standard_normal((2, hq, hd)) * 2.0 ** power).astype(np.float32)
    pos, w = dev(np.array(ctxs, dtype=np.int32) - 1), dev(h.w)
    o = ee.attention_weights(dev(q.reshape(2, -1)), dev(h.k), dev(h.v), dev(h.table), pos, w, hq, hkv, hd, 300)
    o, w, g = o.cpu().numpy().reshape(2, hq, hd), w.cpu().numpy(), np.arange(hq) * hkv // hq
    for s, c in enumerate(ctxs):
        K, V, q64 = h.K[s].astype(np.float64), h.V[s].astype(np.float64), q[s].astype(np.float64)
        z = np.einsum("hd,thd->ht", q64, K[:, g]) / math.sqrt(hd)
        if power > 0:   # the largest score is ahead of the next by more than any error of theirs
            order = np.sort(z, 1)
            assert np.all(order[:, -1] - order[:, -2] > 200 + 2 * score_error(q64, K))
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        # as in check_attention_weights; a one-hot row has no error but its division's
        rel = 0.0 if power > 0 else 2 * score_error(q64, K).max() + 4 * U32 * np.abs(z).max()
        rel += (c + 32) * U32
        ref, mag = np.einsum("ht,thd->hd", p, V[:, g]), np.einsum("ht,thd->hd", p, np.abs(V[:, g]))
        assert np.all(np.abs(o[s] - ref) <= rel * mag + 1e-30), s
        add = np.zeros_like(h.W[s], dtype=np.float64)
        for a in range(hq):
            add[:, g[a]] += p[a]
        assert np.all(np.abs(h.gather(w, s) - h.W[s] - add) <= rel * add + 8 * U32 * (h.W[s] + add)), s


# ------------------------------------------------ faulty lengths and block ids

@pytest.mark.parametrize("bad", [0, 1])
@pytest.mark.parametrize("what", ["block", "negative block", "long", "negative"])
def test_faults_of_one_sequence_leave_the_other_alone(what, bad):
    """With a fault in one sequence every operator reports it, and the other sequence's
    results, its rows and the blocks of no sequence are those of a call without it.  Block
    ids out of range are read as block 0, which here is the good sequence's."""
    hq, hkv, hd = 4, 2, 64
    c = Prompt(51, hq, hkv, hd, [20, 30], [20, 30])
    h, good = c.h, 1 - bad
    # block 0 is the good sequence's first
    at = h.table[good, 0]
    for x in (h.k, h.v, h.w):
        x[[0, at]] = x[[at, 0]]
    h.table[:] = np.where(h.table == 0, -1, np.where(h.table == at, 0, h.table))
    h.table[h.table == -1] = at
    d = c.args()
    own = np.zeros((2, h.n_blocks), dtype=bool)
    for s, n in enumerate(h.ctxs):
        own[s, h.table[s, : (n + 15) // 16]] = True
    rest = dev(~own[bad])   # the good sequence's blocks and those of none
    table, ctx = d["table"].clone(), d["ctx"].clone()
    if "block" in what:
        table[bad, 1] = -3 if "negative" in what else h.n_blocks
    else:
        # whatever is read lies in the cache, and whatever is written in the bad sequence's blocks
        table[bad] = int(h.table[bad, 0])
        ctx[bad] = -5 if what == "negative" else 1 << 30
    decode_q = dev(h.rng.standard_normal((2, hq * hd)).astype(np.float32))
    _, lse = ee.prompt_attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["ctx"], *c.shape)

    def calls(table, ctx):
        err = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(4)]
        res = []
        o, l = ee.prompt_attention(d["q"], d["k"], d["v"], table, d["cu"], ctx, *c.shape, err=err[0])
        rows = c.seq_rows(good)
        res += [o[rows], l[:, rows]]
        w = dev(h.w)
        ee.prompt_weights(d["q"], d["k"], table, d["cu"], ctx, lse, w, *c.shape, err=err[1])
        res.append(w[rest])
        w = dev(h.w)
        x = ee.attention_weights(decode_q, d["k"], d["v"], table, ctx - 1, w, *c.shape, err=err[2])
        res += [x[good], w[rest]]
        k, v, w = d["k"].clone(), d["v"].clone(), dev(h.w)
        kept, new = ee.evict(k, v, w, table, ctx, 7, 2, c.max_ctx, err=err[3])
        res += [kept[good], new[good], k[rest], v[rest], w[rest]]
        return [e.item() for e in err], res

    no_err, want = calls(d["table"], d["ctx"])
    assert no_err == [0] * 4
    errs, got = calls(table, ctx)
    assert errs == [EE_DERR_BLOCK if "block" in what else EE_DERR_LENGTH] * 4
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(bits(a), bits(b)), i


def test_stream_argument():
    """Each operator on a stream that is given: the results of the current one, on that stream."""
    c = Prompt(101, 8, 2, 64, [70, 33], [70, 90])
    d = c.args()
    qd = dev(c.h.rng.standard_normal((2, 512)).astype(np.float32))
    side = torch.cuda.Stream()
    got = []
    for stream in (None, side):
        k, v, w = d["k"].clone(), d["v"].clone(), torch.zeros(c.h.n_blocks, 2, 16, device="cuda")
        torch.cuda.synchronize()
        o, lse = ee.prompt_attention(d["q"], k, v, d["table"], d["cu"], d["ctx"], *c.shape, stream=stream)
        ee.prompt_weights(d["q"], k, d["table"], d["cu"], d["ctx"], lse, w, *c.shape, stream=stream)
        # behind the others on the same stream
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            pos = d["ctx"] - 1
        x = ee.attention_weights(qd, k, v, d["table"], pos, w, *c.shape, stream=stream)
        kept, new = ee.evict(k, v, w, d["table"], d["ctx"], 33, 5, c.max_ctx, stream=stream)
        (stream or torch.cuda.current_stream()).synchronize()
        got.append([o, lse, x, kept, new, k, v, w])
    for a, b in zip(*got):
        assert torch.equal(bits(a), bits(b))
    assert torch.cuda.current_stream() != side


@pytest.mark.parametrize("hq,hkv,hd,ctx", [(8, 2, 64, 200), (8, 8, 128, 1500)])
def test_infinite_scores(hq, hkv, hd, ctx):
    """A score of -infinity weighs nothing, in prompts and decode steps alike; one of +infinity
    makes the rows that see it NaN, with the weights of all tokens that they see."""
    n, G, t = 60, hq // hkv, ctx - 30
    c = Prompt(hq + ctx, hq, hkv, hd, [n], [ctx])
    c.q[:, :, 3] = np.abs(c.q[:, :, 3]) + 0.5
    qd = c.q[-1:].astype(np.float32)
    d, h, off = c.args(), c.h, ctx - n
    at = h.table[0, t // 16], hkv - 1, t % 16, 3

    def call(x):
        k = h.k.copy()
        k[at] = x
        k = dev(k)
        w, wd = (torch.zeros(h.n_blocks, hkv, 16, device="cuda") for _ in range(2))
        o, lse = ee.prompt_attention(d["q"], k, d["v"], d["table"], d["cu"], d["ctx"], *c.shape)
        ee.prompt_weights(d["q"], k, d["table"], d["cu"], d["ctx"], lse, w, *c.shape)
        od = ee.attention_weights(dev(qd.reshape(1, -1)), k, d["v"], d["table"], d["ctx"] - 1, wd, *c.shape)
        w, wd = (h.gather(y.cpu().numpy(), 0).astype(np.float64) for y in (w, wd))
        return o.cpu().numpy().astype(np.float64).reshape(n, hq, hd), lse.cpu().numpy(), w, od.cpu().numpy().reshape(hq, hd), wd

    o, lse, w, od, wd = call(-np.inf)
    K, V = h.K[0].astype(np.float64), h.V[0].astype(np.float64)
    # a score's error twice, the exponential's argument, sums of ctx and n G terms, the division:
    # as in prompt_reference, with the token's key finite
    q64 = c.q.astype(np.float64)
    z = max(np.abs(np.einsum("nhd,thd->nht", q64, K[:, np.arange(hq) // G])).max() / math.sqrt(hd), 1.0)
    rel = 2 * max(score_error(q, K).max() for q in q64) + (ctx + n * G + 40) * U32 + 8 * U32 * z
    K[t, hkv - 1, 3] = -np.inf
    ro, rl, rw = oracle.prompt_attention(q64, K, V)
    # probabilities and result in fp16: half a step each of at most the largest value
    big = np.abs(V).max()
    bo = (2 * 2.0 ** -11 + rel) * big + 2.0 ** -24 * ctx
    assert np.all(np.abs(o - ro) <= bo)
    assert np.all(np.abs(lse - rl) <= rel)
    assert np.all(np.abs(w - rw) <= rel * rw) and np.all(w[t, hkv - 1] == 0)
    rod, _, rw = oracle.prompt_attention(qd.astype(np.float64), K, V)
    assert np.all(np.abs(od - rod[0]) <= rel * big) and np.all(np.abs(wd - rw) <= rel * rw) and wd[t, hkv - 1] == 0

    _, _, w0, od0, wd0 = call(h.k[at])
    o, lse, w, od, wd = call(np.inf)
    g = slice((hkv - 1) * G, hq)   # the heads of the token's kv head
    assert np.isnan(o[t - off:, g]).all() and np.isnan(lse[g, t - off:]).all() and np.isnan(od[g]).all()
    assert np.isnan(w[:, hkv - 1]).all() and np.isnan(wd[:, hkv - 1]).all()   # the last row sees them all
    # Rows before the token do not see it and are what they were, to rounding: a warp goes over
    # to its rows' new maxima for all of them when one's has grown, and an infinite one has.  A
    # probability is off by half a step of fp16 at most whichever maximum it is relative to, so
    # the bounds are the same.
    assert np.all(np.abs(o[: t - off] - ro[: t - off]) <= bo) and np.all(np.abs(lse[:, : t - off] - rl[:, : t - off]) <= rel)
    assert np.array_equal(od[: g.start], od0[: g.start])
    for got, before in ((w, w0), (wd, wd0)):
        assert np.array_equal(got[:, : hkv - 1], before[:, : hkv - 1])


@pytest.mark.parametrize("past", [0, 1800])
@pytest.mark.parametrize("hq,hkv,hd", [(4, 2, 64), (8, 1, 128)])
def test_prompt_attention_values_at_the_end_of_fp16(hq, hkv, hd, past):
    """o is a mean of values, so it is no larger than the largest of them, 65504; where it is
    rounded up on the way it does not become infinite.  Token 0 is ahead of all others so far
    that their exponentials are 0.5 + 0.53 * 2^-11, which fp16 rounds up by 0.47 * 2^-11."""
    n = 99
    c = Prompt(7, hq, hkv, hd, [n], [n + past])
    x = 0.5 + 0.53 * 2.0 ** -11
    ahead = -math.log(x) * math.sqrt(hd)
    c.q[:] = 0
    c.q[..., :2] = 1
    first = np.float16(ahead)
    h = c.h
    for t in range(n + past):
        h.K[0][t] = 0
        h.V[0][t] = 65504
        h.V[0][t, :, 1] = -65504
    h.K[0][0, :, 0], h.K[0][0, :, 1] = first, np.float16(ahead - float(first))
    for t in range(n + past):
        h.k[h.table[0, t // 16], :, t % 16], h.v[h.table[0, t // 16], :, t % 16] = h.K[0][t], h.V[0][t]
    # the score's error, 2^-22 of it and of the residual's rounding, leaves the rounding as it is
    z = (float(first) + float(np.float16(ahead - float(first)))) / math.sqrt(hd)
    assert np.float16(math.exp(-z * (1 + 2.0 ** -20))) == np.float16(math.exp(-z * (1 - 2.0 ** -20))) == np.float16(0.5 + 2.0 ** -11)
    d = c.args()
    o, _ = ee.prompt_attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["ctx"], *c.shape)
    o = o.cpu().numpy().astype(np.float64).reshape(n, hq, hd)
    want = np.full(hd, 65504.0)
    want[1] = -65504.0
    # half a step of fp16 for the probabilities, half a step for o; no value beyond the largest
    assert np.all(np.abs(o) <= 65504) and np.all(np.abs(o - want) <= 2 * 2.0 ** -11 * 65504)
