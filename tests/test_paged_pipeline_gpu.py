"""The dense paged path as a serving loop uses it: prompts admitted and stored, decode steps (live and
recorded) that take pages, write rows and attend, requests that leave and come, next to Quest and SnapKV.
Whole numbers and rows are compared exactly, outputs with the bounds of one rounded probability and one
rounded output, 2^-8 of the weighted value magnitudes and of the result."""
import numpy as np
import pytest
import torch

import oracle.paged as op
import sparse_decode_attention_quest_gb300 as se
from sparse_decode_attention_quest_gb300.pipeline import PagedCache, QuestDecodeStep, SnapKVDecodeCache

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_errors(se_lib, cuda_device):
    se.se_read_device_error(clear=True)
    yield
    assert se.se_read_device_error(clear=True) == 0


def _bf16(shape, g, dev):
    return torch.randn(shape, generator=g).to(torch.bfloat16).to(dev)


def _check_attention(out, lse, k, v, table, lens, q, scale, dv, sink=0, recent=0):
    ref, rlse, mag, zmag = op.decode(k.float().cpu().numpy(), None if v is None else v.float().cpu().numpy(),
                                     table.cpu().numpy(), lens, q.float().cpu().numpy(), scale, dv, sink, recent)
    D = q.shape[-1]
    dz = (D + 8) * 2.0 ** -23 * zmag
    n = np.array(lens)[:, None]
    tol = (2.0 ** -8 + 2 * dz + (n + 64) * 2.0 ** -23)[..., None] * mag + 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7)
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol + 2.0 ** -133).all()
    ltol = dz + (n + 64) * 2.0 ** -23 + 2.0 ** -21 * (1 + np.abs(np.where(np.isinf(rlse), 0, rlse)))
    with np.errstate(invalid="ignore"):
        assert (np.where(np.isneginf(rlse), np.isneginf(lse.cpu().numpy()),
                         np.abs(lse.double().cpu().numpy() - rlse) <= ltol)).all()


SHAPES = {"gqa": dict(num_q_heads=8, num_kv_heads=2, head_dim=128), "wide": dict(num_q_heads=6, num_kv_heads=3, head_dim=256),
          "latent": dict(num_q_heads=16, num_kv_heads=1, head_dim=576, latent=True, head_dim_v=512)}


def _prompts(cache, lens, g, dev, H, D, latent):
    new = torch.tensor(lens, dtype=torch.int32, device=dev)
    cache.extend(new)
    kn = _bf16((sum(lens), H, D), g, dev)
    vn = None if latent else _bf16((sum(lens), H, D), g, dev)
    cache.store(kn, vn)


@pytest.mark.parametrize("shape", list(SHAPES))
def test_recorded_steps_grow_the_cache(cuda_device, shape):
    """One recording of extend + store + attend, replayed over 20 steps: requests cross page borders, one gets no
    token in some steps, and the padded end of the batch of new tokens is skipped."""
    dev, kw = cuda_device, SHAPES[shape]
    Hq, H, D, latent = kw["num_q_heads"], kw["num_kv_heads"], kw["head_dim"], kw.get("latent", False)
    dv = 512 if latent else D
    B, g = 5, torch.Generator().manual_seed(1)
    cache = PagedCache(80, B, 400, max_new_tokens=600, device=dev, **kw)
    lens = [130, 0, 47, 300, 16]
    _prompts(cache, lens, g, dev, H, D, latent)
    assert cache.lens.tolist() == lens
    new = torch.ones(B, dtype=torch.int32, device=dev)
    q = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device=dev)
    kn = torch.zeros(B + 2, H, D, dtype=torch.bfloat16, device=dev)   # two rows of padding
    vn = None if latent else torch.zeros_like(kn)
    stream = torch.cuda.Stream(device=dev)
    torch.cuda.synchronize()
    se.se_capture_begin(stream)
    cache.extend(new, stream)
    cache.store(kn, vn, stream)
    cache.attend(q, stream=stream)
    step = se.se_capture_end(stream)
    assert cache.lens.tolist() == lens  # nothing ran yet
    for t in range(20):
        k_before = cache.k.clone()
        counts = [1, 1, int(t % 3 == 0), 1, 2]
        new.copy_(torch.tensor(counts, dtype=torch.int32))
        q.copy_(_bf16(q.shape, g, dev))
        kn.copy_(_bf16(kn.shape, g, dev))
        if vn is not None:
            vn.copy_(_bf16(vn.shape, g, dev))
        torch.cuda.synchronize()
        step.launch(stream)
        stream.synchronize()
        lens = [a + b for a, b in zip(lens, counts)]
        assert cache.lens.tolist() == lens
        # The rows lie where the slot map says, and nothing else moved.
        slots = cache.slot_map[:sum(counts)].long()
        assert bool((cache.slot_map[sum(counts):] == -1).all())
        k_before[slots // 16, :, slots % 16] = kn[:sum(counts)]
        assert torch.equal(k_before.view(torch.int16), cache.k.view(torch.int16))
        if t % 5 == 4:
            _check_attention(cache.attention.out, cache.attention.lse, cache.k, cache.v, cache.block_table, lens, q,
                             cache.attention.sm_scale, dv)
    step.destroy()
    used = cache.block_table.cpu().numpy()
    pages = [p for b in range(B) for p in used[b, :-(-lens[b] // 16)]]
    assert len(set(pages)) == len(pages) and cache.pool_state.tolist() == [80 - len(pages), 0, 0, 0]


def test_requests_leave_and_others_take_their_pages(cuda_device):
    dev = cuda_device
    g = torch.Generator().manual_seed(2)
    cache = PagedCache(30, 3, 480, 4, 1, 64, 480, dev)
    _prompts(cache, [200, 100, 150], g, dev, 1, 64, False)    # 13 + 7 + 10 pages: all of them
    assert int(cache.pool_state[0]) == 0
    keep = torch.tensor([200, 0, 33], dtype=torch.int32, device=dev)
    cache.release(keep)
    assert cache.lens.tolist() == [200, 0, 33] and int(cache.pool_state[0]) == 14
    _prompts(cache, [8, 170, 15], g, dev, 1, 64, False)
    lens = [208, 170, 48]
    assert cache.lens.tolist() == lens
    q = _bf16((3, 4, 64), g, dev)
    out = cache.attend(q)
    _check_attention(out, cache.attention.lse, cache.k, cache.v, cache.block_table, lens, q, cache.attention.sm_scale, 64)
    out = cache.attend(q, sink_tokens=5, recent_tokens=40)
    _check_attention(out, cache.attention.lse, cache.k, cache.v, cache.block_table, lens, q, cache.attention.sm_scale, 64,
                     5, 40)
    cache.release()
    assert cache.lens.tolist() == [0, 0, 0] and int(cache.pool_state[0]) == 30
    assert sorted(cache.free_pages.tolist()) == list(range(30))
    cache.attend(q)
    assert bool((cache.attention.out == 0).all()) and bool(torch.isneginf(cache.attention.lse).all())


def test_a_stored_cache_serves_the_quest_step(cuda_device):
    """Summaries kept by the row store equal a rebuild, and Quest selecting every page equals dense attention."""
    dev = cuda_device
    g = torch.Generator().manual_seed(3)
    B, Hq, H, D = 3, 16, 2, 128
    cache = PagedCache(140, B, 1024, Hq, H, D, 1200, dev, summary=True)
    lens = [0, 0, 0]
    for chunk in ([500, 31, 0], [123, 400, 17], [1, 1, 1]):   # chunks that begin inside pages
        _prompts(cache, chunk, g, dev, H, D, False)
        lens = [a + b for a, b in zip(lens, chunk)]
    n = cache.lens
    step = QuestDecodeStep(cache.k, cache.v, cache.summary, cache.block_table, Hq, 64, 1024)
    kept = cache.summary.clone()
    step.build_summaries(n)
    used = torch.cat([cache.block_table[b, :-(-lens[b] // 16)] for b in range(B)]).long()
    assert torch.equal(kept[used].view(torch.int16), cache.summary[used].view(torch.int16))
    q = _bf16((B, Hq, D), g, dev)
    sparse = step.run(q, n).clone()
    dense = step.attend_dense(q, n)
    assert bool((step.counts == torch.tensor([-(-x // 16) for x in lens], device=dev, dtype=torch.int32)[:, None]).all())
    _check_attention(dense, step.dense.lse, cache.k, cache.v, cache.block_table, lens, q, step.sm_scale, D)
    assert float((step.dense.lse - step.lse).abs().max()) < 1e-4
    assert float((dense.float() - sparse.float()).abs().max()) < 2e-2


def test_decode_over_a_compacted_cache(cuda_device):
    """A SnapKV-compacted cache through appends and a periodic eviction: the decode attends what is live."""
    dev = cuda_device
    g = torch.Generator().manual_seed(4)
    B, H, Hq, D, W, K, period = 2, 2, 8, 128, 4, 24, 6
    cache = SnapKVDecodeCache(B, H, Hq, D, W, 7, K, 4, 8, period, dev)
    n0 = 90
    pages = 6
    k = _bf16((B * pages, H, 16, D), g, dev)
    v = _bf16((B * pages, H, 16, D), g, dev)
    bt = torch.arange(B * pages, dtype=torch.int32, device=dev).view(B, pages)
    lens = torch.full((B,), n0, dtype=torch.int32, device=dev)
    cache.evict_from(se.paged_kv(k, v, None), bt, lens, _bf16((B, W, Hq, D), g, dev), n0)
    for t in range(2 * period + 1):
        q = _bf16((B, Hq, D), g, dev)
        cache.append(_bf16((B, H, D), g, dev), _bf16((B, H, D), g, dev), q)
        out = cache.attend(q)
        _check_attention(out, cache.attention.lse, cache.k[cache.live], cache.v[cache.live], cache.block_table,
                         cache.lens.tolist(), q, cache.sm_scale, D)
    assert cache.evictions == 3


def test_recordings_of_other_shapes_share_a_workspace(cuda_device):
    """Recorded decodes of other shapes over one workspace, launched one after the other on one stream: joins in
    the decode kernel (narrow tables), in a kernel of their own, and of a latent cache, many of each."""
    dev = cuda_device
    g = torch.Generator().manual_seed(5)
    made = []
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    stream = torch.cuda.Stream(device=dev)
    for Hq, H, D, width, lens in [(8, 2, 128, 4096, [3000, 40]), (4, 1, 64, 1024, [900 + 9 * i for i in range(12)]),
                                  (32, 1, 576, 2048, [700 + 31 * i for i in range(12)])]:
        latent = D == 576
        cache = PagedCache(2000, len(lens), width, Hq, H, D, sum(lens), dev, latent=latent,
                           head_dim_v=512 if latent else None)
        _prompts(cache, lens, g, dev, H, D, latent)
        q = _bf16((len(lens), Hq, D), g, dev)
        cache.attention.workspace = ws
        torch.cuda.synchronize()
        se.se_capture_begin(stream)
        cache.attend(q, stream=stream)
        made.append((cache, q, lens, se.se_capture_end(stream)))
    for _ in range(3):
        for cache, _, _, step in made:
            cache.attention.out.fill_(float("nan"))
            torch.cuda.synchronize()
            step.launch(stream)
            stream.synchronize()
            assert not bool(ws[:768].any())  # the counters are back at zero
    for cache, q, lens, step in made:
        _check_attention(cache.attention.out, cache.attention.lse, cache.k, cache.v, cache.block_table, lens, q,
                         cache.attention.sm_scale, cache.kv.head_dim_v)
        step.destroy()
