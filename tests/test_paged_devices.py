"""The binding of the dense paged path and the device of the cache: the library launches on the current device, so a
cache view of another one is refused like any other tensor there. Fake pointers, never dereferenced."""
import types

import pytest
import torch

import sparse_decode_attention_quest_gb300 as se


def _on(index, *shape, dtype=torch.bfloat16):
    """What the binding looks at of a CUDA tensor on device ``index``."""
    class OnGpu(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return index

    return torch.Tensor._make_subclass(OnGpu, torch.zeros(*shape, dtype=dtype))


@pytest.fixture
def current(monkeypatch):
    """Current device 0 and a library whose calls succeed without running."""
    made = []
    ok = lambda name: lambda *a: made.append(name) or 0
    lib = types.SimpleNamespace(se_paged_kv_store=ok("store"), se_paged_decode=ok("decode"))
    monkeypatch.setattr(se, "load_library", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return made


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("latent", [False, True])
def test_a_cache_on_another_device(current, index, latent):
    D, dv = (576, 512) if latent else (128, 128)
    k = _on(index, 4, 1, 16, D)
    kv = se.paged_kv(k, None if latent else _on(index, 4, 1, 16, D), None, dv)
    rows = _on(0, 2, 1, D)
    store = lambda: se.se_paged_kv_store(kv, rows, None if latent else rows, _on(0, 2, dtype=torch.int32), stream=5)
    decode = lambda: se.se_paged_decode(kv, _on(0, 2, 16, D), _on(0, 2, 3, dtype=torch.int32),
                                        _on(0, 2, dtype=torch.int32), 0.1, _on(0, 2, 16, dv), None,
                                        _on(0, 64, dtype=torch.uint8), stream=5)
    for call in (store, decode):
        if index == 0:
            call()
        else:
            with pytest.raises(ValueError, match="kv: is on cuda:1"):
                call()
    assert current == (["store", "decode"] if index == 0 else [])


def test_a_view_of_the_callers_own_making_is_taken(current):
    k = _on(0, 4, 1, 16, 128)
    kv = se.SEPagedKV(k.data_ptr(), k.data_ptr() + 8, None, 4, 1, 16, 128, 128, 128, 128)
    rows = _on(0, 2, 1, 128)
    se.se_paged_kv_store(kv, rows, rows, _on(0, 2, dtype=torch.int32), stream=5)
    assert current == ["store"]


def test_one_device_for_a_cache():
    k = _on(0, 4, 1, 16, 128)
    assert se.paged_kv(k, _on(0, 4, 1, 16, 128), _on(0, 4, 1, 2, 128)).device == 0
    with pytest.raises(ValueError, match="v_cache: is on cuda:1"):
        se.paged_kv(k, _on(1, 4, 1, 16, 128), None)
    with pytest.raises(ValueError, match="summary: is on cuda:1"):
        se.paged_kv(k, _on(0, 4, 1, 16, 128), _on(1, 4, 1, 2, 128))
