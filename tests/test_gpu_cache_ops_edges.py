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
