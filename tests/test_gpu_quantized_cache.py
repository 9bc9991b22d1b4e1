"""The eight-bit cache through the public entry points: writing against the oracle bit for
bit, reading back, decode attention against 64 bits, and the three as a run."""
import math

import numpy as np
import pytest

import oracle
from tests.cache_cases import U16
from tests.quantized_cases import UNUSED, VALUES, EightBit, attention_reference
from tests.test_gpu_cache_ops import EE_DERR_BLOCK, EE_DERR_LENGTH, dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import early_exit_decoding_layer_gb300 as ee  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from early_exit_decoding_layer_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------ writing

WRITES = [
    # (kv heads, hd, rows, ctxs)
    (1, 64, [1], [1]), (2, 64, [1], [16]), (8, 128, [1, 1, 1], [17, 33, 400]), (2, 128, [40, 0, 7], [40, 9, 50]),
    (3, 64, [5, 31], [5, 100]), (16, 64, [65], [65]), (5, 128, [130, 1], [200, 1]), (2, 64, [9, 4], [3, 0]),
]


def written(rows, ctxs, hkv, hd, dtype, seed=1, lead=1, tail=2, stride=0):
    """A call of quantize_cache, its inputs and the cache that the oracle expects."""
    r = np.random.default_rng(seed + hd + sum(rows))
    cu = np.concatenate([[lead], lead + np.cumsum(rows)]).astype(np.int32)
    T = int(cu[-1]) + tail
    x = r.standard_normal((2, T, hkv, hd)) * np.exp2(r.integers(-20, 14, (2, T, hkv, 1)))
    x[:, :, :, ::7] *= 0.01
    x = x.astype(dtype)
    flat = x.reshape(-1, hd)
    odd = [0.0, -0.0, 448.0, 449.0, 464.0, 2.0 ** -24, 65504.0, -65504.0, np.inf, np.nan, -np.inf, 17.0, 19.0, 240.0]
    for i in range(0, len(flat), 3):
        flat[i, i % hd] = odd[(i // 3) % len(odd)]
    flat[len(flat) // 2] = 0.0
    flat[len(flat) // 2 + 1] = np.nan
    per = max(1, max((c + 15) // 16 for c in ctxs))
    n_blocks = len(ctxs) * per + 2
    table = np.full((len(ctxs), per + 1), UNUSED, dtype=np.int32)
    order = r.permutation(n_blocks)
    codes, exps = np.full((n_blocks, hkv, 2, 16, hd), 0x55, dtype=np.uint8), np.full((n_blocks, hkv, 2, 16), 77, dtype=np.int8)
    want = codes.copy(), exps.copy()
    for s, (n, c) in enumerate(zip(rows, ctxs)):
        first = max(0, c - n) // 16   # entries of tokens before the rows are not read
        nb = (c + 15) // 16
        table[s, first:nb] = order[s * per + first:s * per + nb]
        for i in range(n):
            t = c - n + i
            if t < 0:
                continue
            for kv in range(2):
                for g in range(hkv):
                    at = table[s, t // 16], g, kv, t % 16
                    want[0][at], want[1][at] = oracle.quantize_row(x[kv, cu[s] + i, g])
    wide = [torch.full((T, hkv * hd + stride), 3.0, dtype=torch.from_numpy(x[:1]).dtype, device="cuda") for _ in range(2)]
    for i in range(2):
        wide[i][:, : hkv * hd] = dev(x[i].reshape(T, -1))
    err = i32(0)
    c, e = dev(codes), dev(exps)
    out = ee.quantize_cache(wide[0][:, : hkv * hd], wide[1][:, : hkv * hd], c, e, dev(table), dev(cu), dev(np.array(ctxs, np.int32)),
                            max(max(ctxs), 1) + 3, err=err)
    assert out[0] is c and out[1] is e
    return c.cpu().numpy(), e.cpu().numpy(), want, err.item()


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("hkv,hd,rows,ctxs", WRITES)
def test_quantize_cache(hkv, hd, rows, ctxs, dtype):
    codes, exps, (wc, we), err = written(rows, ctxs, hkv, hd, dtype, stride=8 if len(rows) == 2 else 0)
    assert err == 0
    assert np.array_equal(exps, we)
    nan = (codes & 127) == 127
    assert np.array_equal(nan, (wc & 127) == 127)
    assert np.array_equal(codes[~nan], wc[~nan])


def test_quantize_every_fp16_value():
    """All fp16 values at all exponents that a row can have: bit for bit the oracle's rounding,
    which searches the table of codes."""
    x = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16).view(np.float16)
    big = np.array([2.0 ** -24, 0.0136, 0.0137, 1.0, 448.0, 450.0, 57344.0, 65504.0], dtype=np.float16)
    rows = []
    for b in big:
        fits = x[np.abs(x.astype(np.float64)) <= float(b)]
        fits = np.concatenate([fits, np.zeros(-len(fits) % 63, np.float16)]).reshape(-1, 63)
        rows.append(np.concatenate([np.full((len(fits), 1), b, np.float16), fits], 1))
    rows = np.concatenate(rows)[::5][:16384]
    T = len(rows)
    nb = (T + 15) // 16
    codes = torch.zeros(nb, 1, 2, 16, 64, dtype=torch.float8_e4m3fn, device="cuda")
    exps = torch.zeros(nb, 1, 2, 16, dtype=torch.int8, device="cuda")
    k = dev(rows)
    ee.quantize_cache(k, k, codes, exps, torch.arange(nb, dtype=torch.int32, device="cuda").view(1, -1), i32(0, T), i32(T), T)
    codes, exps = codes.view(torch.uint8).cpu().numpy(), exps.cpu().numpy()
    for kv in range(2):
        got, e = codes[:, 0, kv].reshape(-1, 64)[:T], exps[:, 0, kv].reshape(-1)[:T]
        for i in range(0, T, 17):
            want = oracle.quantize_row(rows[i])
            assert e[i] == want[1] and np.array_equal(got[i], want[0]), i
        held = VALUES[got] * np.exp2(e.astype(np.float64))[:, None]
        # half a step: 2^-4 of a value, and of the least step, 2^-9 codes
        x64 = rows.astype(np.float64)
        assert np.all(np.abs(held - x64) <= np.maximum(2.0 ** -4 * np.abs(x64), 2.0 ** -10 * np.exp2(e.astype(np.float64))[:, None]))


# ------------------------------------------------ reading back

@pytest.mark.parametrize("other", [False, True])
@pytest.mark.parametrize("hkv,hd,ctxs", [(1, 64, [1]), (2, 128, [0, 16, 17]), (8, 64, [700, 33]), (5, 128, [129, 1, 90]), (16, 64, [250])])
def test_dequantize_cache(hkv, hd, ctxs, other):
    h = EightBit(hd + sum(ctxs), ctxs, hkv, hd, scale=-4, spread=11)
    first = h.table[int(np.argmax(ctxs)), 0]
    h.codes[first, 0, 0, 0, :4] = [0x7F, 0xFF, 0x7E, 0xFE]   # NaN, 448
    h.exps[first, 0, 0, 0] = 8
    n_dst = h.n_blocks + 2
    dst = np.full_like(h.table, UNUSED)
    perm = h.rng.permutation(n_dst)
    for s, c in enumerate(ctxs):
        nb = (c + 15) // 16
        dst[s, :nb] = perm[h.table[s, :nb]] if other else h.table[s, :nb]
    k, v = (torch.full((n_dst, hkv, 16, hd), 3.0, dtype=torch.float16, device="cuda") for _ in range(2))
    err = i32(0)
    out = ee.dequantize_cache(dev(h.codes), dev(h.exps), dev(h.table), dev(np.array(ctxs, np.int32)), k, v, max(ctxs) + 2,
                              dst_table=dev(dst) if other else None, err=err)
    assert err.item() == 0 and out[0] is k and out[1] is v
    touched = np.zeros((n_dst, 16), dtype=bool)
    for s, c in enumerate(ctxs):
        t = np.arange(c)
        touched[dst[s, t // 16], t % 16] = True
        K, V, _ = h.history(s)
        for got, want in ((k, K), (v, V)):
            got = got.cpu().numpy()[dst[s, t // 16], :, t % 16]
            assert np.array_equal(got, np.clip(want, -65504, 65504).astype(np.float16), equal_nan=True)
    for x in (k, v):
        assert np.all(np.moveaxis(x.cpu().numpy(), 2, 1)[~touched] == 3.0)


# ------------------------------------------------ decode attention

DECODE = [
    (4, 2, 64, [1]), (4, 2, 64, [0, 15, 16, 17]), (32, 8, 64, [300, 1, 47]), (32, 8, 128, [2304]), (64, 8, 128, [1100, 33]),
    (8, 8, 128, [5, 64, 129, 1000]), (16, 16, 64, [700, 0]), (8, 4, 128, [513, 31]), (4, 1, 64, [5000]), (8, 1, 128, [16384]),
    (2, 1, 64, [127, 128, 129, 255, 256, 257]), (24, 24, 64, [127, 128]), (4, 2, 128, [2]),
]


def check_decode(h, q, hq, table=None, max_ctx=None, codes=None, skip=()):
    B, hkv, hd = len(h.ctxs), h.hkv, h.hd
    err = i32(0)
    o = ee.quantized_attention(dev(q.reshape(B, -1)), dev(h.codes if codes is None else codes), dev(h.exps),
                               dev(h.table if table is None else table), dev(np.array(h.ctxs, np.int32) - 1), hq, hkv, hd,
                               max_ctx or max(max(h.ctxs), 1), err=err)
    assert err.item() == 0
    o = o.cpu().numpy().reshape(B, hq, hd).astype(np.float64)
    for s in range(B):
        if s in skip:
            continue
        want, bound = attention_reference(q[s].astype(np.float64), *h.history(s, codes))
        assert np.all(np.abs(o[s] - want) <= bound), (s, np.max(np.abs(o[s] - want) / bound))
    return o


@pytest.mark.parametrize("hq,hkv,hd,ctxs", DECODE)
def test_quantized_attention(hq, hkv, hd, ctxs):
    h = EightBit(hq + hd + sum(ctxs), ctxs, hkv, hd)
    q = h.rng.standard_normal((len(ctxs), hq, hd)).astype(np.float16)
    check_decode(h, q, hq, max_ctx=min(16384, max(ctxs) + 9))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("hq,hkv,hd,seqs", [(32, 8, 128, 40), (64, 8, 128, 20), (16, 16, 64, 33), (8, 4, 64, 64), (8, 8, 128, 64)])
def test_quantized_attention_many_units(hq, hkv, hd, seqs, wide):
    """More (sequence, kv head) pairs than CTAs; wide: room for 16384 tokens, few of which exist."""
    r = np.random.default_rng(seqs + hd)
    ctxs = [0, 1, 700] + [int(x) for x in np.exp(r.uniform(0, np.log(500), seqs - 3))]
    h = EightBit(hq + seqs, ctxs, hkv, hd)
    q = h.rng.standard_normal((seqs, hq, hd)).astype(np.float16)
    table = np.full((seqs, 1024), UNUSED, dtype=np.int32)
    table[:, : h.table.shape[1]] = h.table
    check_decode(h, q, hq, table, 16384 if wide else max(ctxs))


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("hq,hkv,hd,c", [(8, 1, 128, 1500), (4, 4, 64, 300), (2, 1, 64, 4000)])
def test_quantized_attention_ramps(hq, hkv, hd, c, up):
    """Scores and exponents of V that grow or fall by hundreds along the tokens: the running
    maximum moves all the time."""
    h = EightBit(7, [c], hkv, hd)
    t = np.arange(c)
    at = h.table[0, t // 16], slice(None), slice(None), t % 16
    codes = h.codes[at]
    codes[:, :, 0] = 0
    x = (t / c if up else 1 - t / c) * 400
    codes[:, :, 0, 0] = np.searchsorted(VALUES[:127], x).astype(np.uint8)[:, None]
    h.codes[at] = codes
    e = h.exps[at]
    e[:, :, 0] = -1
    e[:, :, 1] = (-15 + t * 23 // c if up else 8 - t * 23 // c)[:, None]
    h.exps[at] = e
    q = np.zeros((1, hq, hd), dtype=np.float16)
    q[0, :, 0] = np.linspace(-8, 16, hq)
    check_decode(h, q, hq)


def test_quantized_attention_scales():
    """Queries of every size, keys and values at both ends of the exponents."""
    for qs, ek, ev in ((2.0 ** -14, -13, -13), (1.0, -13, 6), (30000.0, -13, 6), (2.0 ** -20, 6, -13), (0.01, 6, 6)):
        h = EightBit(3, [300, 90], 2, 64, scale=ek, spread=2)
        h.exps[:, :, 1] = np.where(np.abs(h.exps[:, :, 1].astype(int)) == 127 + (h.exps[:, :, 1] < 0), h.exps[:, :, 1], ev)
        q = (h.rng.standard_normal((2, 8, 64)) * qs).clip(-65000, 65000).astype(np.float16)
        q[0, 1] = 0
        q[0, 2, 3:] = 0
        check_decode(h, q, 8)


def test_quantized_attention_strided_rows_and_repeat():
    h = EightBit(5, [700, 33, 90], 2, 64)
    q = h.rng.standard_normal((3, 8, 64)).astype(np.float16)
    args = dev(h.codes), dev(h.exps), dev(h.table), i32(699, 32, 89), 8, 2, 64, 700
    ref = ee.quantized_attention(dev(q.reshape(3, -1)), *args)
    wide = torch.full((3, 8 * 64 * 2 + 24), 3.0, dtype=torch.float16, device="cuda")
    wide[:, 8:520] = dev(q.reshape(3, -1))
    for _ in range(20):
        o = ee.quantized_attention(wide[:, 8:520], *args, out=wide[:, 528:1040])
        assert torch.equal(o, ref)
    assert torch.all(wide[:, :8] == 3.0) and torch.all(wide[:, 520:528] == 3.0) and torch.all(wide[:, 1040:] == 3.0)


@pytest.mark.parametrize("hq,hkv,hd,ctxs", [(8, 2, 64, [2100]), (32, 8, 128, [2304, 700]), (4, 4, 128, [290, 600, 33] * 21)])
def test_quantized_attention_nonfinite(hq, hkv, hd, ctxs):
    """A NaN of V reaches its component of the group's heads, a NaN of K or q all of the rows
    that see it, and nothing else changes."""
    h = EightBit(hq + hd + sum(ctxs), ctxs, hkv, hd)
    B, G, c = len(ctxs), hq // hkv, ctxs[0]
    q = h.rng.standard_normal((B, hq, hd)).astype(np.float16)
    args = dev(h.exps), dev(h.table), dev(np.array(ctxs, np.int32) - 1), hq, hkv, hd, max(ctxs)
    call = lambda q, codes: ee.quantized_attention(dev(q.reshape(B, -1)), dev(codes), *args).view(B, hq, hd)  # noqa: E731
    clean = call(q, h.codes)
    assert torch.isfinite(clean).all()
    codes, hit = h.codes.copy(), torch.zeros(B, hq, hd, dtype=torch.bool, device="cuda")
    for (t, g, i) in ((3, 0, 5), (140, hkv - 1, 6), (c - 1, 0, hd - 1), (c - 150, 0, 9)):
        codes[h.table[0, t // 16], g, 1, t % 16, i] = 0x7F
        hit[0, g * G:(g + 1) * G, i] = True
    o = call(q, codes)
    assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], clean[~hit])
    for t in (3, c - 1):
        codes = h.codes.copy()
        codes[h.table[0, t // 16], hkv - 1, 0, t % 16, 8] = 0xFF
        o = call(q, codes)
        hit = torch.zeros(B, hq, dtype=torch.bool, device="cuda")
        hit[0, (hkv - 1) * G:] = True
        assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], clean[~hit])
    for x in (np.nan, np.inf, -np.inf):
        bad = q.copy()
        bad[0, 1, 7] = x
        o = call(bad, h.codes)
        hit = torch.zeros(B, hq, dtype=torch.bool, device="cuda")
        hit[0, 1] = True
        assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], clean[~hit])


def test_quantized_attention_largest_values():
    """Values of 65536 held, whose mean fp16 does not hold: the result is 65504."""
    h = EightBit(9, [200], 1, 64)
    t = np.arange(200)
    at = h.table[0, t // 16], 0, 1, t % 16
    h.codes[at] = 0x78   # 256
    h.codes[at[0], 0, 1, at[3], 32:] = 0xF8
    h.exps[at] = 8
    o = ee.quantized_attention(dev(np.ones((1, 128), np.float16)), dev(h.codes), dev(h.exps), dev(h.table), i32(199), 2, 1, 64, 200)
    o = o.view(2, 64)
    assert torch.all(o[:, :32] == 65504) and torch.all(o[:, 32:] == -65504)


# ------------------------------------------------ together

def test_write_decode_read_run():
    """As they are used: packed prompts written, decode steps that write their token and attend,
    and the cache read back for a chunk of the prompt attention."""
    hq, hkv, hd, rows = 8, 2, 128, [150, 61]
    r = np.random.default_rng(3)
    W = 12
    table = dev(r.permutation(2 * W).astype(np.int32).reshape(2, W))
    codes = torch.zeros(2 * W, hkv, 2, 16, hd, dtype=torch.uint8, device="cuda")
    exps = torch.zeros(2 * W, hkv, 2, 16, dtype=torch.int8, device="cuda")
    kv = [r.standard_normal((2, n + 2, hkv, hd)).astype(np.float16) for n in rows]   # two decode steps behind
    pack = [dev(np.concatenate([x[i, :n] for x, n in zip(kv, rows)]).reshape(sum(rows), -1)) for i in range(2)]
    ctx = dev(np.array(rows, np.int32))
    ee.quantize_cache(*pack, codes, exps, table, i32(0, 150, 211), ctx, 16 * W)
    held = []
    for x in kv:
        c, e = zip(*[oracle.quantize_row(row) for row in x.reshape(-1, hd)])
        held.append((VALUES[np.array(c)] * np.exp2(np.array(e, dtype=np.float64))[:, None]).reshape(x.shape))
    for step in range(2):
        new = [dev(np.stack([x[i, n + step] for x, n in zip(kv, rows)]).reshape(2, -1).astype(np.float32)) for i in range(2)]
        ee.quantize_cache(*new, codes, exps, table, i32(0, 1, 2), ctx + step + 1, 16 * W)
        q = r.standard_normal((2, hq, hd)).astype(np.float16)
        o = ee.quantized_attention(dev(q.reshape(2, -1)), codes, exps, table, ctx + step, hq, hkv, hd, 16 * W)
        e = exps.cpu().numpy().astype(np.float64)
        for s, n in enumerate(rows):
            t = np.arange(n + step + 1)
            ev = e[table.cpu().numpy()[s, t // 16], :, 1, t % 16]
            want, bound = attention_reference(q[s].astype(np.float64), held[s][0, : n + step + 1], held[s][1, : n + step + 1], ev)
            assert np.all(np.abs(o[s].cpu().numpy().reshape(hq, hd) - want) <= bound)
    k, v = (torch.zeros(2 * W, hkv, 16, hd, dtype=torch.float16, device="cuda") for _ in range(2))
    ee.dequantize_cache(codes, exps, table, ctx + 2, k, v, 16 * W)
    chunk = r.standard_normal((7, hq, hd)).astype(np.float16)
    o, _ = ee.prompt_attention(dev(chunk.reshape(7, -1)), k, v, table, i32(0, 4, 7), ctx + 2, hq, hkv, hd, 16 * W)
    for s, n in enumerate(rows):
        part = slice(0, 4) if s == 0 else slice(4, 7)
        want, _, _ = oracle.prompt_attention(chunk[part].astype(np.float64), held[s][0], held[s][1])
        got = o.cpu().numpy().astype(np.float64).reshape(7, hq, hd)[part]
        # fp16 probabilities and result, as in prompt_reference: half a step each of at most the values' size
        assert np.all(np.abs(got - want) <= 2 * U16 * np.abs(held[s][1]).max() + 2.0 ** -24)


def test_capture_replay_and_streams():
    """Two captured runs on two streams, replayed together on changed inputs: each as it is eagerly."""
    runs = []
    for i in range(2):
        ctxs = [[700, 40, 2100], [33, 1500, 900, 16]][i]
        h = EightBit(40 + i, ctxs, 4, 128)
        B = len(ctxs)
        d = dict(q=dev(h.rng.standard_normal((B, 16 * 128)).astype(np.float16)), codes=dev(h.codes), exps=dev(h.exps),
                 table=dev(h.table), ctx=dev(np.array(ctxs, np.int32)), rows=dev(h.rng.standard_normal((2, B, 512)).astype(np.float16)),
                 k=torch.zeros(h.n_blocks, 4, 16, 128, dtype=torch.float16, device="cuda"))
        d["v"] = d["k"].clone()
        cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")

        def run(d=d, cu=cu, most=max(ctxs)):
            ee.quantize_cache(d["rows"][0], d["rows"][1], d["codes"], d["exps"], d["table"], cu, d["ctx"], most)
            o = ee.quantized_attention(d["q"], d["codes"], d["exps"], d["table"], d["ctx"] - 1, 16, 4, 128, most)
            ee.dequantize_cache(d["codes"], d["exps"], d["table"], d["ctx"], d["k"], d["v"], most)
            return o

        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            run()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=stream):
                o = run()
        runs.append((graph, stream, o, d, run))
    for trial in range(3):
        want = []
        for _, _, _, d, run in runs:
            d["rows"].normal_()
            d["q"].normal_()
            want.append((run().clone(), d["k"].clone(), d["v"].clone()))
            d["k"].zero_(), d["v"].zero_()
        torch.cuda.synchronize()
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for (_, _, o, d, _), w in zip(runs, want):
            assert torch.equal(o, w[0]) and torch.equal(d["k"], w[1]) and torch.equal(d["v"], w[2])


def test_bad_lengths_and_blocks_are_reported():
    """The kernels' own checks: the call stays inside the arrays, the error word says what was
    wrong, and sequences without a fault are right."""
    h = EightBit(51, [40, 300], 2, 64)
    q = h.rng.standard_normal((2, 4, 64)).astype(np.float16)
    rows = h.rng.standard_normal((2, 5, 128)).astype(np.float16)
    good = check_decode(h, q, 4, max_ctx=310)

    def calls(table, ctx, cu):
        err = [i32(0) for _ in range(3)]
        c, e = dev(h.codes), dev(h.exps)
        k, v = (torch.zeros(h.n_blocks, 2, 16, 64, dtype=torch.float16, device="cuda") for _ in range(2))
        o = ee.quantized_attention(dev(q.reshape(2, -1)), c, e, table, ctx - 1, 4, 2, 64, 310, err=err[0])
        ee.dequantize_cache(c, e, table, ctx, k, v, 310, err=err[1])
        ee.quantize_cache(dev(rows[0]), dev(rows[1]), c, e, table, cu, ctx, 310, err=err[2])
        return o, [x.item() for x in err]

    cu = i32(0, 2, 5)
    for what, code in (("block", EE_DERR_BLOCK), ("negative block", EE_DERR_BLOCK), ("long", EE_DERR_LENGTH), ("negative", EE_DERR_LENGTH)):
        table, ctx = h.table.copy(), np.array(h.ctxs, np.int32)
        if "block" in what:
            table[0, 2] = -3 if "negative" in what else h.n_blocks
        else:
            ctx[0] = -5 if what == "negative" else 1 << 30
            table[0] = table[1]
            table[0, 19:] = 0
        o, err = calls(dev(table), dev(ctx), cu)
        assert err == [code] * 3, what
        got = o[1].cpu().numpy().reshape(4, 64).astype(np.float64)
        if "block" in what:
            assert np.array_equal(got, good[1]), what
        else:
            # another length moves the borders between the CTAs' shares, so that the same sums are
            # taken in another order: within the bound that holds for every order
            want, bound = attention_reference(q[1].astype(np.float64), *h.history(1))
            assert np.all(np.abs(got - want) <= bound), what
    for bad in ((0, 2, 1 << 30), (-1, 2, 5), (0, 4, 2)):
        assert calls(dev(h.table), dev(np.array(h.ctxs, np.int32)), i32(*bad))[1] == [0, 0, EE_DERR_LENGTH], bad


def test_offsets_beyond_32_bits():
    """Blocks behind 2^32 bytes of codes: the same bits as near the start."""
    hq, hkv, hd = 32, 8, 128
    h = EightBit(71, [200, 70], hkv, hd)
    q = dev(h.rng.standard_normal((2, hq * hd)).astype(np.float16))
    rows = dev(h.rng.standard_normal((2, 2, hkv * hd)).astype(np.float16))
    shift = (1 << 32) // (hkv * 32 * hd) + 1000
    got = []
    for by in (0, shift):
        codes = torch.empty(by + h.n_blocks, hkv, 2, 16, hd, dtype=torch.uint8, device="cuda")
        exps = torch.empty(by + h.n_blocks, hkv, 2, 16, dtype=torch.int8, device="cuda")
        codes[by:], exps[by:] = dev(h.codes), dev(h.exps)
        k, v = (torch.empty(by + h.n_blocks, hkv, 16, hd, dtype=torch.float16, device="cuda") for _ in range(2))
        k[by:], v[by:] = 0, 0
        table = dev(np.where(h.table == UNUSED, h.table, h.table + by))
        ee.quantize_cache(rows[0], rows[1], codes, exps, table, i32(0, 1, 2), i32(200, 70), 200)
        o = ee.quantized_attention(q, codes, exps, table, i32(199, 69), hq, hkv, hd, 200)
        ee.dequantize_cache(codes, exps, table, i32(200, 70), k, v, 200)
        got.append([o] + [x[by:].clone() for x in (codes, exps, k, v)])
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_refusals_on_device_tensors():
    h = EightBit(61, [20], 2, 64)
    ok = dict(q=torch.zeros(1, 256, dtype=torch.float16, device="cuda"), codes=dev(h.codes), exps=dev(h.exps), table=dev(h.table),
              pos=i32(19), shape=(4, 2, 64, 20), out=None)

    def attn(**kw):
        a = {**ok, **kw}
        return ee.quantized_attention(a["q"], a["codes"], a["exps"], a["table"], a["pos"], *a["shape"], out=a["out"])

    attn()
    attn(codes=ok["codes"].view(torch.float8_e4m3fn))
    for kw in (dict(q=ok["q"].float()), dict(q=ok["q"].cpu()), dict(codes=ok["codes"].view(torch.int8)), dict(codes=ok["codes"][:, :, :1]),
               dict(exps=ok["exps"].view(torch.uint8)), dict(exps=ok["exps"][1:]), dict(table=ok["table"].long()), dict(pos=i32(1, 2)),
               dict(out=ok["q"]), dict(out=torch.zeros(1, 255, dtype=torch.float16, device="cuda")), dict(shape=(4, 2, 64, 0)),
               dict(shape=(4, 2, 64, 16385)), dict(shape=(6, 2, 64, 20)), dict(shape=(12, 4, 64, 20))):
        with pytest.raises(ee.EEError) as e:
            attn(**kw)
        assert e.value.status == 1, kw
    k = torch.zeros(4, 128, dtype=torch.float16, device="cuda")
    w = dict(k=k, v=k, codes=ok["codes"], exps=ok["exps"], table=ok["table"], cu=i32(0, 4), ctx=i32(20), max_ctx=20)
    ee.quantize_cache(*w.values())
    for kw in (dict(k=k.bfloat16()), dict(v=k.float()), dict(k=k[:, :120]), dict(v=k[:3]), dict(cu=i32(0)), dict(max_ctx=0),
               dict(k=torch.zeros(4, 132, dtype=torch.float16, device="cuda")[:, :128]), dict(codes=ok["codes"][:, :, :, :8])):
        with pytest.raises(ee.EEError) as e:
            ee.quantize_cache(*{**w, **kw}.values())
        assert e.value.status == 1, kw
    kc, vc = (torch.zeros(h.n_blocks, 2, 16, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    d = dict(codes=ok["codes"], exps=ok["exps"], table=ok["table"], ctx=i32(20), k=kc, v=vc, max_ctx=20, dst=None)
    ee.dequantize_cache(*d.values())
    for kw in (dict(v=kc), dict(k=kc[1:]), dict(k=kc.float()), dict(dst=ok["table"][:, :1]), dict(dst=ok["table"][:0]), dict(ctx=i32(1, 2))):
        with pytest.raises(ee.EEError) as e:
            ee.dequantize_cache(*{**d, **kw}.values())
        assert e.value.status == 1, kw
    torch.cuda.synchronize()


def test_no_rows_is_no_work():
    h = EightBit(63, [20], 2, 64)
    k = torch.zeros(0, 128, dtype=torch.float16, device="cuda")
    codes, exps = dev(h.codes), dev(h.exps)
    ee.quantize_cache(k, k, codes, exps, dev(h.table), i32(0, 0), i32(20), 20)
    assert np.array_equal(codes.cpu().numpy(), h.codes) and np.array_equal(exps.cpu().numpy(), h.exps)


def test_close_to_the_fp16_cache():
    """What eight bits cost: held within half a step (2^-4) of the values, the attention stays
    within what that allows."""
    r = np.random.default_rng(17)
    n, hkv, hd, hq = 500, 2, 128, 8
    x = r.standard_normal((2, n, hkv, hd)).astype(np.float16)
    table = torch.arange(32, dtype=torch.int32, device="cuda").view(1, -1)
    codes = torch.zeros(32, hkv, 2, 16, hd, dtype=torch.uint8, device="cuda")
    exps = torch.zeros(32, hkv, 2, 16, dtype=torch.int8, device="cuda")
    ee.quantize_cache(dev(x[0].reshape(n, -1)), dev(x[1].reshape(n, -1)), codes, exps, table, i32(0, n), i32(n), 512)
    q = r.standard_normal((1, hq, hd)).astype(np.float16)
    o = ee.quantized_attention(dev(q.reshape(1, -1)), codes, exps, table, i32(n - 1), hq, hkv, hd, 512).cpu().numpy().reshape(hq, hd)
    full = oracle.attention_decode(q[0].astype(np.float64), x[0].astype(np.float64), x[1].astype(np.float64))
    for h in range(hq):
        K = np.abs(x[0][:, h // 4].astype(np.float64))
        dz = 2.0 ** -4 * (K @ np.abs(q[0, h].astype(np.float64))).max() / math.sqrt(hd) + 1e-3
        V = np.abs(x[1][:, h // 4].astype(np.float64)).max()
        assert np.all(np.abs(o[h] - full[h]) <= (np.exp(2 * dz) - 1 + 2.0 ** -4 + 2.0 ** -10) * V)
