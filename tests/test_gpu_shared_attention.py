"""Decode attention of a batch that shares a prefix, through the public entry point,
against 64 bits."""
import numpy as np
import pytest

from tests.cache_cases import History, prompt_reference
from tests.test_gpu_cache_ops import EE_DERR_BLOCK, EE_DERR_LENGTH, dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import early_exit_decoding_layer_gb300 as ee  # noqa: E402

UNUSED = 0x7FFFFFF0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from early_exit_decoding_layer_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Shared(History):
    """ctxs[s] tokens of every sequence; all of them begin with the first prefix // 16 blocks of a
    sequence of `prefix` tokens that is in no table but for these."""

    def __init__(self, seed, ctxs, prefix, hkv, hd):
        nb = prefix // 16
        super().__init__(seed, list(ctxs) + [nb * 16], hkv, hd)
        own = self.table[-1, :nb].copy()
        PK, PV = self.K.pop(), self.V.pop()
        self.W.pop()
        self.ctxs = list(ctxs)
        self.table = self.table[:-1].copy()
        self.prefix = prefix
        for s, c in enumerate(ctxs):
            n = min(c, nb * 16)
            self.K[s][:n], self.V[s][:n] = PK[:n], PV[:n]
            # blocks of its own behind the shared ones; entries of shared blocks are row 0's alone
            self.table[s, : min(nb, (c + 15) // 16)] = UNUSED
        most = max((min(c, nb * 16) + 15) // 16 for c in ctxs)
        self.table[0, :most] = own[:most]

    def call(self, q, hq, max_ctx=None, prefix=None, table=None, k=None, v=None, pos=None, **kw):
        B = len(self.ctxs)
        return ee.shared_attention(dev(q.reshape(B, -1)), dev(self.k if k is None else k), dev(self.v if v is None else v),
                                   dev(self.table if table is None else table), dev(np.array(self.ctxs, np.int32) - 1) if pos is None else pos,
                                   self.prefix if prefix is None else prefix, hq, self.hkv, self.hd, max_ctx or max(max(self.ctxs), 1), **kw)

    def check(self, q, hq, **kw):
        err = i32(0)
        o = self.call(q, hq, err=err, **kw).cpu().numpy().astype(np.float64).reshape(q.shape)
        assert err.item() == 0
        for s, c in enumerate(self.ctxs):
            want, _, _, bound, _, _ = prompt_reference(self, s, q[s][None])
            assert np.all(np.abs(o[s] - want[0]) <= bound[0]), (s, np.max(np.abs(o[s] - want[0]) - bound[0]))
        return o


CASES = [
    # (query heads, kv heads, hd, prefix, ctxs)
    (4, 2, 64, 16, [17]), (4, 2, 64, 0, [1, 40, 0]), (8, 2, 128, 33, [34, 50, 64, 33]), (32, 8, 128, 512, [513, 600, 530, 1100]),
    (8, 8, 64, 128, [129] * 5), (8, 1, 128, 130, [131, 300, 144, 145, 160]), (64, 8, 128, 700, [701 + 7 * i for i in range(20)]),
    (16, 16, 64, 256, [257, 1000, 256, 272]), (8, 4, 128, 1000, [1001] * 33), (4, 1, 64, 5000, [5001, 5200]),
    # 129 rows, 256, 257, 512 of a kv head
    (8, 1, 64, 300, [301 + i for i in range(17)]), (8, 1, 64, 300, [301 + i for i in range(32)]), (8, 1, 128, 200, [210] * 33),
    (16, 2, 128, 400, [401 + 3 * i for i in range(64)]), (1, 1, 64, 64, [65 + i for i in range(64)]),
    # sequences that end within the prefix, some empty ones, the first too
    (8, 2, 64, 200, [250, 100, 0, 192, 193, 7, 200]), (8, 4, 128, 320, [0, 400, 16, 1]), (4, 2, 64, 320, [100, 50, 319]),
    # tails longer than the prefix
    (32, 8, 128, 64, [2000, 70, 900]), (8, 2, 64, 16, [3000, 17]),
]


@pytest.mark.parametrize("hq,hkv,hd,prefix,ctxs", CASES)
def test_shared_attention(hq, hkv, hd, prefix, ctxs):
    h = Shared(hq + hd + prefix, ctxs, prefix, hkv, hd)
    q = h.rng.standard_normal((len(ctxs), hq, hd)).astype(np.float16)
    h.check(q, hq)
    h.check(q, hq, max_ctx=min(16384, 16 * h.table.shape[1]))


@pytest.mark.parametrize("hq,hkv,hd", [(32, 8, 128), (64, 8, 64)])
def test_long_prefix(hq, hkv, hd):
    """Near the largest length, with tails of every size, and table columns that are not used."""
    ctxs = [15001, 15400, 16384, 15017, 15008]
    h = Shared(3, ctxs, 15000, hkv, hd)
    q = h.rng.standard_normal((len(ctxs), hq, hd)).astype(np.float16)
    q[:, :, 0] += 3   # some tokens weigh much
    h.check(q, hq, max_ctx=16384)


@pytest.mark.parametrize("hq,hkv,hd,prefix,most", [(64, 8, 128, 1000, 400), (64, 8, 64, 520, 300), (32, 8, 128, 700, 500), (16, 16, 64, 300, 700)])
def test_many_units(hq, hkv, hd, prefix, most):
    """64 sequences: row tiles of all sizes, and CTAs that go through many sequences' own tiles, one
    or few each, behind a share of the prefix; the same bits every time."""
    rng = np.random.default_rng(hq + hd)
    ctxs = [prefix + int(x) for x in np.exp(rng.uniform(0, np.log(most), 64))]
    ctxs[5], ctxs[20], ctxs[63] = 0, prefix // 2, prefix // 16 * 16
    h = Shared(11, ctxs, prefix, hkv, hd)
    q = h.rng.standard_normal((64, hq, hd)).astype(np.float16)
    h.check(q, hq)
    args = (dev(q.reshape(64, -1)), dev(h.k), dev(h.v), dev(h.table), dev(np.array(ctxs, np.int32) - 1), prefix, hq, hkv, hd, max(ctxs))
    err, first = i32(0), None
    for _ in range(20):
        o = ee.shared_attention(*args, err=err)
        first = o if first is None else first
        assert torch.equal(o, first)
    assert err.item() == 0


def test_prefix_behind_the_longest_sequence():
    """A prefix longer than max_ctx: as much of it as there is."""
    h = Shared(4, [100, 40], 112, 2, 64)
    q = h.rng.standard_normal((2, 8, 64)).astype(np.float16)
    h.check(q, 8, max_ctx=100)


@pytest.mark.parametrize("hq,hkv,hd,prefix,ctxs", [(8, 2, 64, 600, [601, 900, 640]), (32, 8, 128, 0, [300, 2000]), (8, 8, 128, 48, [50] * 40)])
def test_agrees_with_each_alone(hq, hkv, hd, prefix, ctxs):
    """The prefix's length changes how it is computed and not what: no prefix, parts of it."""
    h = Shared(5, ctxs, prefix, hkv, hd)
    table = h.table.copy()
    table[:, : prefix // 16] = table[0, : prefix // 16]
    q = h.rng.standard_normal((len(ctxs), hq, hd)).astype(np.float16)
    for p in {0, min(16, prefix), prefix // 2, prefix}:
        h.check(q, hq, prefix=p, table=table)


def test_strided_rows_and_repeat():
    h = Shared(6, [700, 333, 390, 320], 320, 2, 64)
    q = h.rng.standard_normal((4, 8, 64)).astype(np.float16)
    ref = h.call(q, 8)
    wide = torch.full((4, 8 * 64 * 2 + 24), 3.0, dtype=torch.float16, device="cuda")
    wide[:, 8:520] = dev(q.reshape(4, -1))
    for _ in range(20):
        o = ee.shared_attention(wide[:, 8:520], dev(h.k), dev(h.v), dev(h.table), i32(699, 332, 389, 319), 320, 8, 2, 64, 700,
                                out=wide[:, 528:1040])
        assert torch.equal(o, ref)
    assert torch.all(wide[:, :8] == 3.0) and torch.all(wide[:, 520:528] == 3.0) and torch.all(wide[:, 1040:] == 3.0)


@pytest.mark.parametrize("up", [False, True])
def test_sharp_rows(up):
    """Scores that grow or fall by hundreds along the tokens, in the prefix and behind it."""
    n = 900
    h = Shared(7, [n, 700, 640], 640, 1, 64)
    q = np.zeros((3, 4, 64), dtype=np.float16)
    q[:, :, 0] = [8.0, -8.0, 1.0, 0.0]
    ramp = (np.arange(n) * 0.25 * (1 if up else -1)).astype(np.float16)
    full = h.table.copy()
    full[:, :40] = full[0, :40]
    for s, c in enumerate(h.ctxs):
        for t in range(c):
            h.K[s][t] = 0
            h.K[s][t, 0, 0] = ramp[t]
            h.k[full[s, t // 16], 0, t % 16] = h.K[s][t, 0]
    h.check(q, 4)


def test_nonfinite():
    """A value that is not finite reaches the rows that see its token, in its own component; a NaN key
    all of them; a sequence that ends before it none."""
    hq, hkv, hd, ctxs = 8, 2, 64, [500, 200, 340, 0, 321]
    h = Shared(8, ctxs, 320, hkv, hd)
    q = h.rng.standard_normal((len(ctxs), hq, hd)).astype(np.float16)
    clean = h.call(q, hq).view(len(ctxs), hq, hd)
    assert torch.isfinite(clean).all()
    full = h.table.copy()
    full[:, :20] = np.where(full[:, :20] == UNUSED, full[0, :20], full[:, :20])
    sees = lambda t, s: [x for x, c in enumerate(ctxs) if c > t and (t < 320 or x == s)]  # noqa: E731
    cells = {(3, 0, 0, 5): np.inf, (210, 0, 1, 6): np.nan, (319, 0, 0, 40): -np.inf, (499, 0, 1, 9): np.inf, (330, 2, 0, 63): np.nan}
    v, hit = h.v.copy(), torch.zeros(clean.shape, dtype=torch.bool, device="cuda")
    for (t, s, g, i), x in cells.items():
        v[full[s, t // 16], g, t % 16, i] = x
        for r in sees(t, s):
            hit[r, g * 4:(g + 1) * 4, i] = True
    o = h.call(q, hq, v=v).view(clean.shape)
    assert not torch.isfinite(o[hit]).any() and torch.equal(o[~hit], clean[~hit])
    for t, s in ((3, 0), (250, 0), (320, 0), (339, 2)):
        k = h.k.copy()
        k[full[s, t // 16], 1, t % 16, 8] = np.nan
        hit = torch.zeros(clean.shape[:2], dtype=torch.bool, device="cuda")
        hit[sees(t, s), 4:] = True
        o = h.call(q, hq, k=k).view(clean.shape)
        assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], clean[~hit]), t
    # scores of -infinity alone: nothing weighs
    bad = q.copy()
    bad[1, 2, 3] = np.nan
    o = h.call(bad, hq).view(clean.shape)
    hit = torch.zeros(clean.shape[:2], dtype=torch.bool, device="cuda")
    hit[1, 2] = True
    assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], clean[~hit])


def test_largest_values():
    """Values of 65504 whose probabilities round up: the result stays finite."""
    h = Shared(9, [300, 128], 128, 1, 64)
    h.v[:] = np.where(np.isnan(h.v), h.v, np.float16(65504))
    q = h.rng.standard_normal((2, 8, 64)).astype(np.float16)
    o = h.call(q, 8)
    assert torch.isfinite(o).all() and torch.all(o >= 65504 * (1 - 2.0 ** -10))


def test_capture_replay_and_streams():
    """Two captured calls on two streams, replayed together on changed inputs."""
    runs = []
    for i in range(2):
        h = Shared(40 + i, [[900, 40 + 640, 2100], [700, 661, 650, 641]][i], 640, 4, 128)
        B = len(h.ctxs)
        d = dict(q=dev(h.rng.standard_normal((B, 16 * 128)).astype(np.float16)), k=dev(h.k), v=dev(h.v), table=dev(h.table),
                 pos=dev(np.array(h.ctxs, np.int32) - 1))
        run = lambda d=d, most=max(h.ctxs): ee.shared_attention(d["q"], d["k"], d["v"], d["table"], d["pos"], 640, 16, 4, 128, most)  # noqa: E731
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
            d["q"].normal_()
            want.append(run().clone())
        torch.cuda.synchronize()
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for (_, _, o, _, _), w in zip(runs, want):
            assert torch.equal(o, w)


def test_bad_lengths_and_blocks_are_reported():
    h = Shared(51, [400, 360, 340], 320, 2, 64)
    q = h.rng.standard_normal((3, 4, 64)).astype(np.float16)
    good = h.call(q, 4, max_ctx=410)
    for what, code in (("block", EE_DERR_BLOCK), ("negative block", EE_DERR_BLOCK), ("long", EE_DERR_LENGTH), ("negative", EE_DERR_LENGTH)):
        table, pos = h.table.copy(), np.array(h.ctxs, np.int32) - 1
        if "block" in what:
            table[1, 21] = -3 if "negative" in what else h.n_blocks
        else:
            pos[1] = -5 if what == "negative" else (1 << 31) - 1
            table[1, 20:] = 0
        err = i32(0)
        o = h.call(q, 4, max_ctx=410, table=table, pos=dev(pos), err=err)
        assert err.item() == code, what
        for s in (0, 2):
            if "block" in what:
                assert torch.equal(o[s], good[s]), what
            else:
                # another length moves the borders between the CTAs' shares, so that the same sums
                # are taken in another order: within the bound that holds for every order
                want, _, _, bound, _, _ = prompt_reference(h, s, q[s][None])
                assert np.all(np.abs(o[s].cpu().numpy().astype(np.float64).reshape(4, 64) - want[0]) <= bound[0]), what
    table = h.table.copy()
    table[0, 3] = h.n_blocks   # of the prefix
    err = i32(0)
    h.call(q, 4, table=table, err=err)
    assert err.item() == EE_DERR_BLOCK


def test_offsets_beyond_32_bits():
    hq, hkv, hd = 32, 8, 128
    h = Shared(71, [200, 170], 144, hkv, hd)
    q = h.rng.standard_normal((2, hq, hd)).astype(np.float16)
    near = h.call(q, hq)
    shift = (1 << 32) // (hkv * 16 * hd) + 1000
    k, v = (torch.empty(shift + h.n_blocks, hkv, 16, hd, dtype=torch.float16, device="cuda") for _ in range(2))
    k[shift:], v[shift:] = dev(h.k), dev(h.v)
    table = dev(np.where(h.table == UNUSED, h.table, h.table + shift))
    far = ee.shared_attention(dev(q.reshape(2, -1)), k, v, table, i32(199, 169), 144, hq, hkv, hd, 200)
    assert torch.equal(near, far)


def test_refusals_on_device_tensors():
    h = Shared(61, [40], 16, 2, 64)
    q = torch.zeros(1, 256, dtype=torch.float16, device="cuda")
    ok = dict(q=q, k=dev(h.k), v=dev(h.v), table=dev(h.table), pos=i32(39), prefix=16, shape=(4, 2, 64, 40), out=None)

    def attn(**kw):
        a = {**ok, **kw}
        return ee.shared_attention(a["q"], a["k"], a["v"], a["table"], a["pos"], a["prefix"], *a["shape"], out=a["out"])

    attn()
    for kw in (dict(q=q.float()), dict(q=q.cpu()), dict(k=ok["k"][:, :, :, :32]), dict(v=ok["v"][1:]), dict(table=ok["table"].long()),
               dict(pos=i32(1, 2)), dict(out=q), dict(out=torch.zeros(2, 256, dtype=torch.float16, device="cuda")), dict(prefix=-1),
               dict(prefix=16385), dict(shape=(4, 2, 64, 0)), dict(shape=(4, 2, 64, 16385)), dict(shape=(6, 2, 64, 20))):
        with pytest.raises(ee.EEError) as e:
            attn(**kw)
        assert e.value.status == 1, kw
    with pytest.raises(TypeError):
        attn(prefix=1.5)
    torch.cuda.synchronize()
