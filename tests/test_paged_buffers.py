"""Host side of the dense paged path's buffers: a step's calls only launch. What they need is made when the step
is, so that its fills are not left on another stream than the call's, nor inside a recording."""
import contextlib

import pytest
import torch
from torch.overrides import TorchFunctionMode

import sparse_decode_attention_quest_gb300 as se
from sparse_decode_attention_quest_gb300 import pipeline


@pytest.fixture
def calls(monkeypatch, se_lib):
    """Steps on CPU tensors, whose se_paged_decode calls are recorded instead of made."""
    made = []

    def kv(k, v, summary, head_dim_v=None):
        P, H, page, D = k.shape
        return se.SEPagedKV(k.data_ptr(), (k if v is None else v).data_ptr(), None, P, H, page, D,
                            head_dim_v if v is None else D, D, D)

    monkeypatch.setattr(pipeline, "paged_kv", kv)
    monkeypatch.setattr(pipeline, "se_paged_decode",
                        lambda kv, q, table, lens, scale, out, lse, ws, sink, recent, stream: made.append((ws, stream)))
    return made


def _no_new_buffers(monkeypatch):
    for name in ("empty", "zeros", "full", "arange"):
        def refuse(*args, _name=name, **kw):
            raise AssertionError(f"torch.{_name} in a call")
        monkeypatch.setattr(torch, name, refuse)


@pytest.mark.parametrize("latent", [False, True])
def test_attend_dense_makes_no_buffers(calls, monkeypatch, latent):
    D, Hq = (576, 16) if latent else (128, 8)
    k = torch.zeros(6, 1, 16, D, dtype=torch.bfloat16)
    step = pipeline.QuestDecodeStep(k, None if latent else k.clone(), pipeline.new_summary(k),
                                    torch.zeros(2, 3, dtype=torch.int32), Hq, 4, 48, head_dim_v=512 if latent else None)
    q, lens = torch.zeros(2, Hq, D, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    _no_new_buffers(monkeypatch)
    for stream in (11, 12):
        assert step.attend_dense(q, lens, stream=stream) is step.dense.out
    assert [s for _, s in calls] == [11, 12] and all(ws is step.dense.workspace for ws, _ in calls)
    assert not bool(step.dense.workspace.any())


def test_attend_over_a_compacted_cache_makes_no_buffers(calls, monkeypatch):
    cache = pipeline.SnapKVDecodeCache(2, 2, 8, 128, 4, 7, 24, 4, 8, 6, "cpu")
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    _no_new_buffers(monkeypatch)
    for stream in (11, 12):
        assert cache.attend(q, stream=stream) is cache.attention.out
    assert [s for _, s in calls] == [11, 12] and all(ws is cache.attention.workspace for ws, _ in calls)


class _Ops(TorchFunctionMode):
    """Names of torch's calls, with the stream that was current for each."""

    def __init__(self):
        self.seen, self.current = [], None

    def __torch_function__(self, func, types, args=(), kwargs=None):
        self.seen.append((getattr(func, "__name__", ""), self.current))
        return func(*args, **(kwargs or {}))

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s if s is not None else self.current
        try:
            yield
        finally:
            self.current = before


def test_a_compacted_cache_keeps_to_the_calls_stream(calls, monkeypatch):
    """append and evict_from compute lengths and keep queries with torch: on the stream that their kernels use."""
    cache = pipeline.SnapKVDecodeCache(2, 2, 8, 128, 4, 7, 24, 4, 8, 6, "cpu")
    rows, q = torch.zeros(2, 2, 128, dtype=torch.bfloat16), torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    ops, mine = _Ops(), object()
    monkeypatch.setattr(torch.cuda, "stream", ops.stream)
    for name in ("se_quest_update_summaries", "se_snapkv_score_and_compact_windowed"):
        monkeypatch.setattr(pipeline, name, lambda *a, **kw: None)
    monkeypatch.setattr(pipeline, "se_snapkv_workspace_size", lambda *a: 64)
    with ops:
        for _ in range(cache.period):
            cache.append(rows, rows, q, stream=mine)
    assert cache.evictions == 1
    work = [(name, s) for name, s in ops.seen if name in ("add", "__add__", "copy_", "contiguous", "empty", "zeros")]
    assert {name for name, _ in work} >= {"copy_", "contiguous", "empty"} and len(work) >= cache.period + 6
    assert all(s is mine for _, s in work)
