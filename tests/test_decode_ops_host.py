"""Argument checks of the eight-bit cache's operators and of the shared-prefix attention through
the C ABI and the binding, and the oracle of eight bits: CPU only, every call here is
refused before any CUDA call."""
import math
import types

import numpy as np
import pytest

import early_exit_decoding_layer_gb300 as ee
import oracle


@pytest.fixture(scope="module")
def lib():
    from early_exit_decoding_layer_gb300 import build
    build.build()
    return ee.load_library()


def quantize_cache(lib, **kw):
    a = dict(n_seqs=1, total=4, n_kv_heads=2, head_dim=64, max_ctx=64, rows_type=0, k=16, k_stride=128, v=32, v_stride=128, codes=16,
             exps=16, n_blocks=4, table=16, stride=4, cu=16, ctx=16, err=None)
    a.update(kw)
    return lib.ee_op_quantize_cache(*a.values(), None)


def dequantize_cache(lib, **kw):
    a = dict(n_seqs=1, n_kv_heads=2, head_dim=64, max_ctx=64, codes=16, exps=16, n_blocks=4, table=16, stride=4, ctx=16, k=16, v=32,
             n_dst=4, dst=None, dst_stride=0, err=None)
    a.update(kw)
    return lib.ee_op_dequantize_cache(*a.values(), None)


def quantized_attention(lib, **kw):
    a = dict(n_seqs=1, n_heads=4, n_kv_heads=2, head_dim=64, max_ctx=64, q=16, q_stride=256, codes=16, exps=16, n_blocks=4, table=16,
             stride=4, pos=16, o=32, o_stride=256, scratch=16, err=None)
    a.update(kw)
    return lib.ee_op_quantized_attention(*a.values(), None)


def shared_attention(lib, **kw):
    a = dict(n_seqs=1, n_heads=4, n_kv_heads=2, head_dim=64, max_ctx=64, prefix=16, q=16, q_stride=256, k=16, v=16, n_blocks=4, table=16,
             stride=4, pos=16, o=32, o_stride=256, scratch=16, err=None)
    a.update(kw)
    return lib.ee_op_shared_attention(*a.values(), None)


CACHE = [dict(n_seqs=0), dict(n_seqs=65), dict(n_kv_heads=0), dict(head_dim=96), dict(max_ctx=0), dict(max_ctx=16385), dict(n_blocks=0),
         dict(n_blocks=1 << 27), dict(table=None), dict(table=2), dict(stride=0)]
EIGHT = [dict(codes=None), dict(codes=8), dict(exps=None), dict(exps=8)]
DECODE = [dict(n_heads=0), dict(n_heads=5), dict(n_heads=6), dict(n_heads=32), dict(q=None), dict(q=8), dict(q_stride=248),
          dict(q_stride=260), dict(o=None), dict(o=8), dict(o=16), dict(o_stride=252), dict(pos=None), dict(pos=2), dict(scratch=None),
          dict(scratch=8)]


@pytest.mark.parametrize("kw", CACHE + EIGHT + [dict(total=-1), dict(total=(1 << 24) + 1), dict(rows_type=2), dict(rows_type=-1), dict(k=None),
                                                dict(k=8), dict(v=None), dict(v=8), dict(k_stride=120), dict(v_stride=132),
                                                dict(rows_type=1, k_stride=130), dict(cu=None), dict(ctx=2)], ids=str)
def test_quantize_cache_refuses(lib, kw):
    assert quantize_cache(lib, **kw) == 1


@pytest.mark.parametrize("kw", CACHE + EIGHT + [dict(ctx=None), dict(k=None), dict(k=8), dict(v=None), dict(v=16), dict(n_dst=0),
                                                dict(n_dst=1 << 27), dict(dst=2, dst_stride=4), dict(dst=16, dst_stride=0),
                                                dict(dst=16, dst_stride=3)], ids=str)
def test_dequantize_cache_refuses(lib, kw):
    assert dequantize_cache(lib, **kw) == 1


@pytest.mark.parametrize("kw", CACHE + EIGHT + DECODE, ids=str)
def test_quantized_attention_refuses(lib, kw):
    assert quantized_attention(lib, **kw) == 1


@pytest.mark.parametrize("kw", CACHE + DECODE + [dict(k=None), dict(k=8), dict(v=None), dict(v=8), dict(prefix=-1), dict(prefix=16385)], ids=str)
def test_shared_attention_refuses(lib, kw):
    assert shared_attention(lib, **kw) == 1


def test_no_rows_is_no_work(lib):
    assert quantize_cache(lib, total=0, k=None, v=None) == 0


def test_scratch_sizes(lib):
    for f, more in ((lib.ee_quantized_attention_scratch_bytes, ()), (lib.ee_shared_attention_scratch_bytes, (512,))):
        assert f(1, 4, 2, 64, 100, *more) > 0 and f(64, 64, 8, 128, 16384, *more) > 0
        for bad in ((0, 4, 2, 64, 100), (65, 4, 2, 64, 100), (1, 6, 2, 64, 100), (1, 4, 2, 96, 100), (1, 4, 2, 64, 0), (1, 4, 2, 64, 16385)):
            assert f(*bad, *more) == 0
    assert lib.ee_shared_attention_scratch_bytes(1, 4, 2, 64, 100, -1) == 0


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    q = torch.zeros(2, 256, dtype=torch.float16)
    codes, exps = torch.zeros(4, 2, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2, 2, 16, dtype=torch.int8)
    k = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: ee.quantize_cache(q, q, codes, exps, i.view(1, 2), i, i[:1], 32),
                 lambda: ee.dequantize_cache(codes, exps, i.view(1, 2), i[:1], k, k, 32),
                 lambda: ee.quantized_attention(q, codes, exps, i.view(1, 2), i[:1], 4, 2, 64, 32),
                 lambda: ee.shared_attention(q, k, k, i.view(1, 2), i[:1], 16, 4, 2, 64, 32),
                 lambda: ee.quantize_cache(q, None, codes, exps, i.view(1, 2), i, i[:1], 32),
                 lambda: ee.shared_attention([1.0], k, k, i, i, 16, 4, 2, 64, 32)):
        with pytest.raises(ee.EEError) as e:
            call()
        assert e.value.status == 1


CALLS = {"quantize_cache": 8, "dequantize_cache": 7, "quantized_attention": 9, "shared_attention": 10}


@pytest.mark.parametrize("name", CALLS)
def test_stream_of_another_device_is_refused(name, monkeypatch):
    torch = pytest.importorskip("torch")
    x = types.SimpleNamespace(device=torch.device("cuda", 1))
    streams = [types.SimpleNamespace(device=torch.device("cuda", i)) for i in range(2)]
    used = []

    class Current:
        def __init__(self, stream):
            used.append(stream)

        def __enter__(self):
            return self

        def __exit__(self, *exc):
            return False

    monkeypatch.setattr(torch.cuda, "stream", Current)
    monkeypatch.setattr(ee, "_cache_ops", lambda: types.SimpleNamespace(**{name: lambda *a: "called"}))
    call = getattr(ee, name)
    with pytest.raises(ee.EEError) as e:
        call(*[x] * CALLS[name], stream=streams[0])
    assert e.value.status == 1 and not used
    assert call(*[x] * CALLS[name], stream=streams[1]) == "called" and used == [streams[1]]


def test_oracle_e4m3_table():
    v = oracle.e4m3_values()
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[56] == 1 and v[126] == 448 and math.isnan(v[127]) and math.isnan(v[255])
    assert np.array_equal(v[128:255], -v[:127]) and np.all(np.diff(v[:127]) > 0)


def test_oracle_e4m3_table_is_torch_s():
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, oracle.e4m3_values(), equal_nan=True)


def test_oracle_quantize_row():
    codes, e = oracle.quantize_row([1.0, -448.0, 17.0, 19.0, 0.0, -0.0, np.nan])
    # 17 lies between 16 and 18, 19 between 18 and 20: ties to the even code
    assert e == 0 and codes.tolist() == [56, 254, 88, 90, 0, 128, 127]
    assert oracle.quantize_row([448.5])[1] == 1 and oracle.quantize_row([449.0, np.inf])[1] == 1
    assert oracle.quantize_row([0.0])[1] == -15 and oracle.quantize_row([np.nan, np.inf])[0].tolist() == [127, 127]
    assert oracle.quantize_row([65504.0]) == (np.array([0x78]), 8) and oracle.quantize_row([65520.0])[0][0] == 127
    assert oracle.quantize_row([2.0 ** -24])[0][0] == 1
