"""The dense paged path on a stream of its own, while the current stream is busy with something else, and first
calls inside a recording. The results are compared bit for bit with those of the current stream."""
import pytest
import torch

import sparse_decode_attention_quest_gb300 as se
from sparse_decode_attention_quest_gb300.pipeline import PAGE, QuestDecodeStep, SnapKVDecodeCache, new_summary

pytestmark = pytest.mark.gpu

BUSY = 400_000_000  # clocks: a fifth of a second


@pytest.fixture(autouse=True)
def _no_device_errors(se_lib, cuda_device):
    se.se_read_device_error(clear=True)
    yield
    assert se.se_read_device_error(clear=True) == 0


def _bf16(shape, g, dev):
    return torch.randn(shape, generator=g).to(torch.bfloat16).to(dev)


def _equal(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def _step(dev, latent, seed=1):
    """A Quest step over two requests, one of them split over many CTAs."""
    g = torch.Generator().manual_seed(seed)
    H, Hq, D = (1, 16, 576) if latent else (2, 8, 128)
    width = 600
    k = _bf16((2 * width, H, PAGE, D), g, dev)
    v = None if latent else _bf16((2 * width, H, PAGE, D), g, dev)
    table = torch.randperm(2 * width, generator=g).view(2, width).int().to(dev)
    lens = torch.tensor([9001, 300], dtype=torch.int32, device=dev)
    make = lambda: QuestDecodeStep(k, v, new_summary(k), table, Hq, 4, 16 * width, head_dim_v=512 if latent else None)
    return make, _bf16((2, Hq, D), g, dev), lens


@pytest.mark.parametrize("latent", [False, True])
def test_first_dense_call_on_a_side_stream(cuda_device, latent):
    make, q, lens = _step(cuda_device, latent)
    want = make().attend_dense(q, lens).clone()
    # Memory that the next step's workspace may get, with no zero in it.
    junk = torch.full((64 << 20,), 0xAB, dtype=torch.uint8, device=cuda_device)
    del junk
    step = make()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    out = step.attend_dense(q, lens, stream=s)
    s.synchronize()
    with torch.cuda.stream(s):
        assert _equal(out, want)
    torch.cuda.synchronize()
    assert _equal(step.attend_dense(q, lens), want)


@pytest.mark.parametrize("latent", [False, True])
def test_first_dense_call_in_a_recording(cuda_device, latent):
    make, q, lens = _step(cuda_device, latent)
    want = make().attend_dense(q, lens).clone()
    step = make()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    se.se_capture_begin(s)
    step.attend_dense(q, lens, stream=s)
    graph = se.se_capture_end(s)
    for _ in range(2):
        step.dense.out.fill_(7.0)
        torch.cuda.synchronize()
        graph.launch(s)
        s.synchronize()
        assert _equal(step.dense.out, want)
    graph.destroy()
    assert _equal(step.attend_dense(q, lens), want)


def test_first_call_over_a_compacted_cache_on_a_side_stream(cuda_device):
    dev, g = cuda_device, torch.Generator().manual_seed(2)
    B, H, Hq, D, W, n = 2, 2, 8, 128, 4, 3000
    pages = -(-n // PAGE)
    k, v = _bf16((B * pages, H, PAGE, D), g, dev), _bf16((B * pages, H, PAGE, D), g, dev)
    table = torch.arange(B * pages, dtype=torch.int32, device=dev).view(B, pages)
    lens = torch.full((B,), n, dtype=torch.int32, device=dev)
    window, q = _bf16((B, W, Hq, D), g, dev), _bf16((B, Hq, D), g, dev)

    def make():
        cache = SnapKVDecodeCache(B, H, Hq, D, W, 7, 2500, 4, 8, 6, dev)
        cache.evict_from(se.paged_kv(k, v, None), table, lens, window, n)
        return cache

    want = make().attend(q).clone()
    cache = make()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    out = cache.attend(q, stream=s)
    s.synchronize()
    with torch.cuda.stream(s):
        assert _equal(out, want)


@pytest.mark.parametrize("as_handle", [False, True])
def test_steps_of_a_compacted_cache_on_a_side_stream(cuda_device, as_handle):
    """Appends, the periodic evictions and the attention between them, none of it on the busy current stream."""
    dev, g = cuda_device, torch.Generator().manual_seed(3)
    B, H, Hq, D, W, n, period = 2, 2, 8, 128, 4, 90, 6
    pages = -(-n // PAGE)
    k, v = _bf16((B * pages, H, PAGE, D), g, dev), _bf16((B * pages, H, PAGE, D), g, dev)
    table = torch.arange(B * pages, dtype=torch.int32, device=dev).view(B, pages)
    lens = torch.full((B,), n, dtype=torch.int32, device=dev)
    window = _bf16((B, W, Hq, D), g, dev)
    rows = [(_bf16((B, H, D), g, dev), _bf16((B, H, D), g, dev), _bf16((B, Hq, D), g, dev))
            for _ in range(2 * period + 1)]

    def steps(stream):
        cache = SnapKVDecodeCache(B, H, Hq, D, W, 7, 24, 4, 8, period, dev)
        torch.cuda.synchronize()
        if stream is not None:
            torch.cuda._sleep(BUSY)
        given = stream.cuda_stream if as_handle and stream is not None else stream
        outs = []
        with torch.cuda.stream(stream):
            copies = [torch.empty(B, Hq, D, dtype=torch.bfloat16, device=dev) for _ in rows]
        cache.evict_from(se.paged_kv(k, v, None), table, lens, window, n, given)
        for (kn, vn, q), copy in zip(rows, copies):
            cache.append(kn, vn, q, given)
            out = cache.attend(q, given)
            with torch.cuda.stream(stream):
                outs.append(copy.copy_(out))
        if stream is not None:
            stream.synchronize()
        torch.cuda.synchronize()
        assert cache.evictions == 3
        return outs, cache.lens.tolist()

    want, n_want = steps(None)
    got, n_got = steps(torch.cuda.Stream())
    assert n_got == n_want and all(_equal(a, b) for a, b in zip(got, want))


def test_steps_of_a_compacted_cache_refuse_to_be_recorded(cuda_device):
    """Before anything is recorded or changed; the recording and the cache go on."""
    dev, g = cuda_device, torch.Generator().manual_seed(4)
    B, H, Hq, D = 2, 2, 8, 128
    cache = SnapKVDecodeCache(B, H, Hq, D, 4, 7, 24, 4, 8, 6, dev)
    kn, vn, q = _bf16((B, H, D), g, dev), _bf16((B, H, D), g, dev), _bf16((B, Hq, D), g, dev)
    k = _bf16((B, H, PAGE, D), g, dev)
    table, lens = torch.arange(B, dtype=torch.int32, device=dev).view(B, 1), torch.full((B,), 16, dtype=torch.int32, device=dev)
    window = _bf16((B, 4, Hq, D), g, dev)
    cache.append(kn, vn, q)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for given in (s, s.cuda_stream):
        se.se_capture_begin(s)
        with pytest.raises(RuntimeError, match="recorded"):
            cache.append(kn, vn, q, given)
        with pytest.raises(RuntimeError, match="recorded"):
            cache.evict_from(se.paged_kv(k, k, None), table, lens, window, 16, given)
        cache.attend(q, given)
        graph = se.se_capture_end(s)
        assert cache.steps == 1 and cache.evictions == 0 and cache.lens.tolist() == [1, 1]
        cache.attention.out.fill_(7.0)
        torch.cuda.synchronize()
        graph.launch(s)
        s.synchronize()
        # One token: its weight is 1.
        assert _equal(cache.attention.out, vn.repeat_interleave(Hq // H, 1))
        graph.destroy()
    cache.append(kn, vn, q, s)
    s.synchronize()
    with torch.cuda.stream(s):
        assert cache.lens.tolist() == [2, 2]
