"""The cache operators' argument checks through the C ABI and the binding, and their
64-bit oracle: CPU only, every call here is refused before any CUDA call."""
import math

import numpy as np
import pytest

import early_exit_decoding_layer_gb300 as ee
import oracle


@pytest.fixture(scope="module")
def lib():
    from early_exit_decoding_layer_gb300 import build
    build.build()
    return ee.load_library()


def prompt_attention(lib, **kw):
    a = dict(n_seqs=1, total_q=4, n_heads=4, n_kv_heads=2, head_dim=64, max_ctx=64, q=256, q_stride=256, k=16, v=16, n_blocks=4,
             table=16, stride=4, cu=16, ctx=16, o=512, o_stride=256, lse=16, err=None)
    a.update(kw)
    return lib.ee_op_prompt_attention(*a.values(), None)


def prompt_weights(lib, **kw):
    a = dict(n_seqs=1, total_q=4, n_heads=4, n_kv_heads=2, head_dim=64, max_ctx=64, q=256, q_stride=256, k=16, n_blocks=4,
             table=16, stride=4, cu=16, ctx=16, lse=16, weights=16, err=None)
    a.update(kw)
    return lib.ee_op_prompt_weights(*a.values(), None)


def attention_weights(lib, **kw):
    a = dict(B=1, n_heads=4, n_kv_heads=2, head_dim=64, max_ctx=64, q=16, k=16, v=16, n_blocks=4, table=16, stride=4, pos=16,
             o=16, weights=16, err=None)
    a.update(kw)
    return lib.ee_op_attention_weights(*a.values(), None)


def evict(lib, **kw):
    a = dict(B=1, n_kv_heads=2, head_dim=64, max_ctx=64, keep=8, recent=2, k=16, v=16, weights=16, n_blocks=4, table=16,
             stride=4, dst=None, dst_stride=0, ctx=16, new_ctx=32, kept=16, err=None)
    a.update(kw)
    return lib.ee_op_evict(*a.values(), None)


CACHE = [dict(n_kv_heads=0), dict(head_dim=96), dict(max_ctx=0), dict(max_ctx=16385), dict(k=None), dict(k=8),
         dict(n_blocks=0), dict(n_blocks=1 << 27), dict(table=None), dict(table=2), dict(stride=0)]
GROUP = [dict(n_heads=0), dict(n_heads=5), dict(n_heads=6), dict(n_heads=32)]
ROWS = [dict(n_seqs=0), dict(n_seqs=65), dict(total_q=-1), dict(total_q=(1 << 24) + 1), dict(q=None), dict(q=8),
        dict(q_stride=248), dict(q_stride=260), dict(cu=None), dict(ctx=None)]


@pytest.mark.parametrize("kw", CACHE + GROUP + ROWS + [dict(v=None), dict(o=None), dict(o=8), dict(o=256), dict(o_stride=252),
                                                       dict(lse=2)], ids=str)
def test_prompt_attention_refuses(lib, kw):
    assert prompt_attention(lib, **kw) == 1


@pytest.mark.parametrize("kw", CACHE + GROUP + ROWS + [dict(lse=None), dict(weights=None), dict(weights=4)], ids=str)
def test_prompt_weights_refuses(lib, kw):
    assert prompt_weights(lib, **kw) == 1


@pytest.mark.parametrize("kw", CACHE + GROUP + [dict(B=0), dict(B=65), dict(q=None), dict(q=8), dict(v=None), dict(pos=None),
                                                dict(o=None), dict(weights=None)], ids=str)
def test_attention_weights_refuses(lib, kw):
    assert attention_weights(lib, **kw) == 1


@pytest.mark.parametrize("kw", CACHE + [dict(B=0), dict(B=65), dict(keep=0), dict(keep=16385), dict(recent=-1), dict(recent=9),
                                        dict(weights=None), dict(weights=24), dict(ctx=None), dict(new_ctx=None), dict(new_ctx=16), dict(kept=2),
                                        dict(dst=16, dst_stride=0), dict(dst=16, dst_stride=1, keep=17), dict(dst=2)], ids=str)
def test_evict_refuses(lib, kw):
    assert evict(lib, **kw) == 1


def test_no_rows_is_no_work(lib):
    assert prompt_attention(lib, total_q=0, q=None, o=None) == 0
    assert prompt_weights(lib, total_q=0, q=None, lse=None) == 0


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    q = torch.zeros(2, 256, dtype=torch.float16)
    k = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: ee.prompt_attention(q, k, k, i.view(1, 2), i, i[:1], 4, 2, 64, 32),
                 lambda: ee.prompt_weights(q, k, i.view(1, 2), i, i[:1], q, q, 4, 2, 64, 32),
                 lambda: ee.attention_weights(q.float(), k, k, i.view(1, 2), i[:1], q, 4, 2, 64, 32),
                 lambda: ee.evict(k, k, q, i.view(1, 2), i[:1], 1, 0, 32)):
        with pytest.raises(ee.EEError) as e:
            call()
        assert e.value.status == 1


def test_binding_refuses_what_is_no_tensor_or_integer():
    torch = pytest.importorskip("torch")
    q = torch.zeros(2, 256, dtype=torch.float16)
    for call in (lambda: ee.prompt_attention([1.0], q, q, q, q, q, 4, 2, 64, 32), lambda: ee.evict(None, q, q, q, q, 1, 0, 32)):
        with pytest.raises(ee.EEError) as e:
            call()
        assert e.value.status == 1


def test_error_codes_match_header():
    import os
    import re
    from tests.conftest import ROOT
    src = open(os.path.join(ROOT, "include", "ee.h")).read()
    assert re.search(r"EE_DERR_LENGTH = 16, EE_DERR_BLOCK = 17", src)


def test_oracle_prompt_attention_closed_forms():
    # equal scores: the mean of the visible values, lse = log of their number
    V = np.arange(12, dtype=np.float64).reshape(4, 1, 3)
    o, lse, w = oracle.prompt_attention(np.zeros((3, 2, 3)), np.ones((4, 1, 3)), V)
    for i, n in enumerate((2, 3, 4)):
        assert np.allclose(o[i], V[:n, 0].mean(0)) and np.allclose(lse[:, i], math.log(n))
    assert np.allclose(w[:, 0], [2 * (1 / 2 + 1 / 3 + 1 / 4), 2 * (1 / 2 + 1 / 3 + 1 / 4), 2 * (1 / 3 + 1 / 4), 2 / 4])
    # the last row is the single-token attention
    rng = np.random.default_rng(1)
    q, K, V = rng.standard_normal((5, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    assert np.allclose(oracle.prompt_attention(q, K, V)[0][-1], oracle.attention_decode(q[-1], K, V))
    # rows before the first token see nothing; every row that sees something gives 1
    o, lse, w = oracle.prompt_attention(q, K[:3], V[:3])
    assert np.all(o[:2] == 0) and np.all(np.isneginf(lse[:, :2])) and np.isclose(w.sum(), 3 * 4)


def test_oracle_evict_indices():
    w = np.array([[3.0], [1.0], [np.nan], [1.0], [5.0], [0.0]])
    assert oracle.evict_indices(w, 4, 1).tolist() == [[0, 1, 4, 5]]   # of the two ones the first
    assert oracle.evict_indices(w, 2, 2).tolist() == [[4, 5]]
    assert oracle.evict_indices(w, 5, 0).tolist() == [[0, 1, 3, 4, 5]]
    assert oracle.evict_indices(w, 6, 0).tolist() == [list(range(6))]
