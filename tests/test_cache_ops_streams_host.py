"""The cache operators refuse a stream of another device than their tensors': CPU only, with
stand-ins for both."""
import types

import pytest

import early_exit_decoding_layer_gb300 as ee

torch = pytest.importorskip("torch")

CALLS = {"prompt_attention": 10, "prompt_weights": 11, "attention_weights": 10, "evict": 8}


@pytest.mark.parametrize("name", CALLS)
def test_stream_of_another_device_is_refused(name, monkeypatch):
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
