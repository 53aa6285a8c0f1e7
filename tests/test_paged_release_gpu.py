"""Lengths after a release that is refused, in part or as a whole."""
import numpy as np
import pytest
import torch

import sparse_decode_attention_quest_gb300 as se
from sparse_decode_attention_quest_gb300.pipeline import PagedCache

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_errors(se_lib, cuda_device):
    se.se_read_device_error(clear=True)
    yield
    assert se.se_read_device_error(clear=True) == 0


def _i32(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _cache(dev, lens):
    cache = PagedCache(40, len(lens), 320, 4, 1, 64, 600, dev)
    cache.extend(_i32(lens, dev))
    return cache


def test_a_refused_request_keeps_its_length(cuda_device):
    cache = _cache(cuda_device, [40, 20, 100, 7])
    cache.release(_i32([41, 3, -1, 2**31 - 1], cuda_device))
    assert se.se_read_device_error(clear=True) == se.DEVERR_LENGTH
    assert cache.lens.tolist() == [40, 3, 100, 7]
    assert cache.pool_state.tolist() == [40 - (3 + 1 + 7 + 1), 0, 0, 0]
    # What is left can still be given back, every page once.
    cache.release()
    assert cache.lens.tolist() == [0, 0, 0, 0]
    assert sorted(cache.free_pages.tolist()) == list(range(40))


def test_a_refused_release_keeps_every_length(cuda_device):
    """More pages than the pool lacks: nothing comes back, and nothing shrinks."""
    cache = _cache(cuda_device, [40, 20])
    cache.pool_state[0] = 38
    free = cache.free_pages.clone()
    cache.release(_i32([3, 0], cuda_device))
    assert se.se_read_device_error(clear=True) == se.DEVERR_PAGE_RANGE
    assert cache.lens.tolist() == [40, 20]
    assert torch.equal(free, cache.free_pages) and cache.pool_state.tolist() == [38, 0, 0, 0]


def test_a_recorded_release_serves_refused_and_granted_lengths(cuda_device):
    cache = _cache(cuda_device, [40, 20, 100])
    keep = _i32([0, 0, 0], cuda_device)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    se.se_capture_begin(stream)
    cache.release(keep, stream)
    step = se.se_capture_end(stream)
    assert cache.lens.tolist() == [40, 20, 100]
    for wanted, left, err in [([33, 21, 100], [33, 20, 100], se.DEVERR_LENGTH), ([32, 0, 17], [32, 0, 17], 0),
                              ([1, 1, 1], [1, 0, 1], se.DEVERR_LENGTH)]:
        keep.copy_(_i32(wanted, cuda_device))
        torch.cuda.synchronize()
        step.launch(stream)
        stream.synchronize()
        assert se.se_read_device_error(clear=True) == err
        assert cache.lens.tolist() == left
        assert int(cache.pool_state[0]) == 40 - sum(-(-n // 16) for n in left)
    step.destroy()


@pytest.mark.parametrize("batch", [1, 33, 700, 16384])
@pytest.mark.parametrize("target", ["other", "seq_lens", "keep_lens"])
def test_lengths_after(cuda_device, batch, target):
    """Many requests, some refused, into a buffer of their own and over either input."""
    dev, g = cuda_device, np.random.default_rng(batch)
    width, lens = 3, g.integers(0, 49, batch)
    keep = g.integers(-4, 53, batch)
    keep = np.where(g.random(batch) < 0.3, lens, keep)
    lens[g.random(batch) < 0.05] = 49                     # more than the table holds
    fine = (keep >= 0) & (keep <= lens) & (lens <= 48)
    first, last = -(-np.maximum(keep, 0) // 16), np.minimum(-(-lens // 16), width)
    back = [b * width + p for b in range(batch) if fine[b] for p in range(first[b], last[b])]
    free = torch.full((batch * width,), -9, dtype=torch.int32, device=dev)
    state, table = _i32([0, 0, 0, 0], dev), torch.arange(batch * width, dtype=torch.int32, device=dev).view(batch, width)
    n, k = _i32(lens, dev), _i32(keep, dev)
    after = {"other": torch.full_like(n, -9), "seq_lens": n, "keep_lens": k}[target]
    se.se_block_tables_release_ex(free, state, table, n, k, after)
    assert se.se_read_device_error(clear=True) == (0 if fine.all() else se.DEVERR_LENGTH)
    assert after.tolist() == np.where(fine, keep, lens).tolist()
    assert state.tolist() == [len(back), 0, 0, 0] and free[:len(back)].tolist() == back[::-1]
    for name, t, was in [("seq_lens", n, lens), ("keep_lens", k, keep)]:
        assert name == target or t.tolist() == was.tolist()


def test_every_token_by_default(cuda_device):
    dev = cuda_device
    cache = _cache(dev, [40, 20, 100, 7])
    after = torch.full((4,), -9, dtype=torch.int32, device=dev)
    se.se_block_tables_release_ex(cache.free_pages, cache.pool_state, cache.block_table, cache.lens, None, after)
    assert after.tolist() == [0, 0, 0, 0] and cache.lens.tolist() == [40, 20, 100, 7]
    assert cache.free_pages.tolist() == list(range(40)) and int(cache.pool_state[0]) == 40
    for bad, kind in [(after[:3], ValueError), (after.float(), TypeError), (None, TypeError)]:
        with pytest.raises(kind):
            se.se_block_tables_release_ex(cache.free_pages, cache.pool_state, cache.block_table, cache.lens, None, bad)
