"""Calls of the eight-bit cache's operators and of the shared-prefix attention that their
documentation allows and other tests do not make: the most kv heads and sequences, the
first call of a process under capture, both attentions at the same time, graphs that
share a memory pool, one cache read in two ways, a single block."""
import subprocess
import sys

import numpy as np
import pytest

from tests.cache_cases import U16, prompt_reference
from tests.conftest import ROOT
from tests.quantized_cases import EightBit, attention_reference
from tests.test_gpu_cache_ops import dev
from tests.test_gpu_quantized_cache import check_decode
from tests.test_gpu_shared_attention import Shared

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


MOST = [
    # (query heads, kv heads, hd)
    (1024, 1024, 64), (2048, 256, 128), (4096, 512, 64), (1024, 1024, 128),
]


@pytest.mark.parametrize("hq,hkv,hd", MOST)
def test_most_heads_and_sequences_quantized(hq, hkv, hd):
    r = np.random.default_rng(hkv + hd)
    ctxs = [int(x) for x in r.integers(0, 40, 64)]
    ctxs[63] = 39
    h = EightBit(hq, ctxs, hkv, hd)
    q = h.rng.standard_normal((64, hq, hd)).astype(np.float16)
    a = check_decode(h, q, hq, max_ctx=300, skip=set(range(64)) - {0, 31, 32, 63})
    assert np.all(a[[s for s in range(64) if ctxs[s] == 0]] == 0)
    assert np.array_equal(a, check_decode(h, q, hq, max_ctx=300, skip=set(range(64))))
    # read back, and written again: the codes that were there
    k, v = (torch.zeros(h.n_blocks, hkv, 16, hd, dtype=torch.float16, device="cuda") for _ in range(2))
    pos = dev(np.array(ctxs, np.int32))
    ee.dequantize_cache(dev(h.codes), dev(h.exps), dev(h.table), pos, k, v, 300)
    rows = [np.concatenate([x.cpu().numpy()[h.table[s, np.arange(c) // 16], :, np.arange(c) % 16] for s, c in enumerate(ctxs)])
            for x in (k, v)]
    cu = np.concatenate([[0], np.cumsum(ctxs)]).astype(np.int32)
    codes, exps = torch.zeros_like(dev(h.codes)), torch.zeros_like(dev(h.exps))
    ee.quantize_cache(*[dev(x.reshape(len(x), -1)) for x in rows], codes, exps, dev(h.table), dev(cu), pos, 300)
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    ee.dequantize_cache(codes, exps, dev(h.table), pos, k2, v2, 300)
    # held values are held again as they are: a coarser exponent would have to lose a bit of the
    # largest one, and it is the least that holds it
    assert torch.equal(k, k2) and torch.equal(v, v2)


@pytest.mark.parametrize("hq,hkv,hd", MOST)
def test_most_heads_and_sequences_shared(hq, hkv, hd):
    r = np.random.default_rng(hkv + hd)
    ctxs = [int(x) for x in r.integers(0, 60, 64)]
    ctxs[0], ctxs[63] = 33, 59
    h = Shared(hq, ctxs, 32, hkv, hd)
    q = h.rng.standard_normal((64, hq, hd)).astype(np.float16)
    o = h.call(q, hq, max_ctx=300)
    assert torch.equal(o, h.call(q, hq, max_ctx=300))
    o = o.cpu().numpy().astype(np.float64).reshape(q.shape)
    for s in (0, 31, 32, 63):
        want, _, _, bound, _, _ = prompt_reference(h, s, q[s][None])
        assert np.all(np.abs(o[s] - want[0]) <= bound[0])
    assert np.all(o[[s for s in range(64) if ctxs[s] == 0]] == 0)


def test_first_calls_may_be_captured():
    """The first call of each operator in a process, made while a stream is captured."""
    code = """
import torch
import early_exit_decoding_layer_gb300 as ee
d = "cuda"
k, v = (torch.randn(20, 128, device=d).half() for _ in range(2))
q = torch.randn(1, 256, device=d).half()
codes, exps = torch.zeros(4, 2, 2, 16, 64, dtype=torch.uint8, device=d), torch.zeros(4, 2, 2, 16, dtype=torch.int8, device=d)
kc, vc = (torch.zeros(4, 2, 16, 64, device=d).half() for _ in range(2))
t = torch.arange(4, dtype=torch.int32, device=d).view(1, 4)
cu, n = torch.tensor([0, 20], dtype=torch.int32, device=d), torch.tensor([20], dtype=torch.int32, device=d)
pos = n - 1
torch.cuda.synchronize()
g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(g, stream=s):
    ee.quantize_cache(k, v, codes, exps, t, cu, n, 64)
    o = ee.quantized_attention(q, codes, exps, t, pos, 4, 2, 64, 64)
    ee.dequantize_cache(codes, exps, t, n, kc, vc, 64)
    x = ee.shared_attention(q, kc, vc, t, pos, 16, 4, 2, 64, 64)
g.replay()
torch.cuda.synchronize()
assert o.abs().max() > 0 and torch.allclose(x, o, atol=5e-3), (x - o).abs().max()
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ok" in r.stdout, r.stderr[-2000:]


def states():
    """The two attentions over caches that hold the same values."""
    hq, hkv, hd, ctxs = 16, 4, 128, [700, 513, 900, 2100, 515]
    h = Shared(9, ctxs, 512, hkv, hd)
    full = h.table.copy()
    full[:, :32] = full[0, :32]
    B = len(ctxs)
    cu = np.concatenate([[0], np.cumsum(ctxs)]).astype(np.int32)
    rows = [dev(np.concatenate(x).reshape(cu[-1], -1)) for x in (h.K, h.V)]
    codes = torch.zeros(h.n_blocks, hkv, 2, 16, hd, dtype=torch.uint8, device="cuda")
    exps = torch.zeros(h.n_blocks, hkv, 2, 16, dtype=torch.int8, device="cuda")
    table, pos = dev(full), dev(np.array(ctxs, np.int32) - 1)
    for s in range(B):   # shared blocks: one sequence after another, the same values again
        ee.quantize_cache(*[x[cu[s]:cu[s + 1]] for x in rows], codes, exps, table[s:s + 1].contiguous(), i32(0, ctxs[s]),
                          i32(ctxs[s]), 2100)
    k, v = (torch.zeros(h.n_blocks, hkv, 16, hd, dtype=torch.float16, device="cuda") for _ in range(2))
    ee.dequantize_cache(codes, exps, table, pos + 1, k, v, 2100)
    q = dev(h.rng.standard_normal((B, hq * hd)).astype(np.float16))
    quantized = lambda: ee.quantized_attention(q, codes, exps, table, pos, hq, hkv, hd, 2100)   # noqa: E731
    shared = lambda: ee.shared_attention(q, k, v, table, pos, 512, hq, hkv, hd, 2100)           # noqa: E731
    return q, v, quantized, shared


def test_one_history_read_in_two_ways():
    """The eight-bit cache as it is, and read back behind a shared prefix: one answer."""
    _, v, quantized, shared = states()
    # both of the same held values: fp16 results (half a step each) and probabilities (fp16; 12 bits)
    assert (quantized().double() - shared().double()).abs().max().item() <= (3 * U16 + 2.0 ** -12) * v.abs().max().item()


def test_both_attentions_at_once():
    """On two streams, and as branches of one graph whose memory comes from one pool."""
    q, _, quantized, shared = states()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    want = quantized(), shared()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        with torch.cuda.stream(a):
            x = quantized()
        with torch.cuda.stream(b):
            y = shared()
        got.append((x, y))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, want[0]) and torch.equal(y, want[1])
    g, h = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=a):
        b.wait_stream(a)
        x = quantized()
        with torch.cuda.stream(b):
            y = shared()
        z = quantized()
        a.wait_stream(b)
    with torch.cuda.graph(h, stream=a, pool=g.pool()):
        w = shared()
    for _ in range(3):
        q.normal_()
        want = quantized().clone(), shared().clone()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want[0]) and torch.equal(y, want[1]) and torch.equal(z, want[0])
        h.replay()
        torch.cuda.synchronize()
        assert torch.equal(w, want[1])


@pytest.mark.parametrize("n", [1, 15, 16])
def test_a_single_block(n):
    """A cache of one block, which all sequences read, and a table of one column."""
    hq, hkv, hd = 8, 2, 64
    one = EightBit(n, [n], hkv, hd, spare=0, extra_cols=0)
    q = one.rng.standard_normal((3, hq, hd)).astype(np.float16)
    table, pos = i32(0, 0, 0).view(3, 1), i32(n - 1, 0, -1)
    o = ee.quantized_attention(dev(q.reshape(3, -1)), dev(one.codes), dev(one.exps), table, pos, hq, hkv, hd, 16384)
    k, v = (torch.zeros(1, hkv, 16, hd, dtype=torch.float16, device="cuda") for _ in range(2))
    ee.dequantize_cache(dev(one.codes), dev(one.exps), table, pos + 1, k, v, 16384)
    x = ee.shared_attention(dev(q.reshape(3, -1)), k, v, table, pos, 16384, hq, hkv, hd, 16384)
    K, V, ev = one.history(0)
    for s, c in enumerate([n, 1, 0]):
        want, bound = attention_reference(q[s].astype(np.float64), K[:c], V[:c], ev[:c])
        assert np.all(np.abs(o[s].cpu().numpy().reshape(hq, hd) - want) <= bound)
        # of fp16 probabilities: another half step of the values
        bound = bound + 2 * U16 * (np.abs(V[:c]).max() if c else 0.0)
        assert np.all(np.abs(x[s].cpu().numpy().reshape(hq, hd) - want) <= bound)
