"""The write of ragged batches of new rows on the GPU against a token-by-token simulation. Rows are
copies and bounds are minima and maxima of bf16 values: every comparison is exact."""
import numpy as np
import pytest
import torch

import oracle.paged as op
import sparse_decode_attention_quest_gb300 as se

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_errors(se_lib, cuda_device):
    se.se_read_device_error(clear=True)
    yield
    assert se.se_read_device_error(clear=True) == 0


def _bf16(shape, g):
    return torch.randn(shape, generator=g).to(torch.bfloat16)


def _slots(runs, g):
    """Slot map of requests holding ``before`` tokens and getting ``new``, pages handed out at random."""
    pages = sum(-(-(b + n) // 16) for b, n in runs)
    perm = torch.randperm(pages, generator=g).tolist()
    slots, at = [], 0
    for b, n in runs:
        slots += [perm[at + (b + i) // 16] * 16 + (b + i) % 16 for i in range(n)]
        at += -(-(b + n) // 16)
    return slots, max(pages, 1)


def _check(dev, slots, pages, H, D, Dv=None, summary=True, latent=False, fused=0, pad_k=0, pad_v=0, seed=0, err=0):
    g = torch.Generator().manual_seed(seed)
    Dv = D if Dv is None else Dv
    T = len(slots)
    k = _bf16((pages, H, 16, D + pad_k), g)
    v = None if latent else _bf16((pages, H, 16, Dv + pad_v), g)
    s = None
    if summary:
        s = torch.cat([_bf16((pages, H, 1, D), g) - 1, _bf16((pages, H, 1, D), g) + 1], 2).contiguous()
    # Rows as columns of a wider tensor when ``fused`` (more heads before and behind them).
    kn = _bf16((T, fused + H + fused, D), g)
    vn = None if latent else _bf16((T, fused + H + fused, Dv), g)
    dk, dvv, ds = k.to(dev), None if v is None else v.to(dev), None if s is None else s.to(dev)
    kv = se.paged_kv(dk, dvv, ds, Dv)
    kv.head_dim = D            # padded rows: the cache tensors' last dim is the row stride
    kv.head_dim_v = Dv
    dkn, dvn = kn.to(dev), None if vn is None else vn.to(dev)
    args = (kv, dkn[:, fused:fused + H], None if vn is None else dvn[:, fused:fused + H],
            torch.tensor(slots, dtype=torch.int32, device=dev))
    se.se_paged_kv_store(*args)
    assert se.se_read_device_error(clear=True) == err
    nk, ns = k.float().numpy(), None if s is None else s.float().numpy()
    nv = None if v is None else v.float().numpy()
    op.store(nk[..., :D], None if nv is None else nv[..., :Dv], ns, kn.float().numpy()[:, fused:fused + H],
             None if vn is None else vn.float().numpy()[:, fused:fused + H], slots)
    np.testing.assert_array_equal(dk.float().cpu().numpy(), nk)
    if v is not None:
        np.testing.assert_array_equal(dvv.float().cpu().numpy(), nv)
    if s is not None:
        np.testing.assert_array_equal(ds.float().cpu().numpy(), ns)
        se.se_paged_kv_store(*args)   # the same rows again change nothing
        assert se.se_read_device_error(clear=True) == err
        np.testing.assert_array_equal(ds.float().cpu().numpy(), ns)


RUNS = {
    "one": [(0, 1)], "one_inside": [(5, 1)], "page": [(0, 16)], "over_a_border": [(9, 13)], "long": [(3, 200)],
    "decode": [(i * 7, 1) for i in range(40)], "ragged": [(0, 33), (15, 1), (16, 1), (31, 66), (7, 9), (0, 1), (48, 16)],
    "many": [(i % 19, 1 + (i * i) % 45) for i in range(90)],
}


@pytest.mark.parametrize("runs", list(RUNS))
@pytest.mark.parametrize("summary", [True, False])
@pytest.mark.parametrize("H,D", [(4, 128), (1, 64)])
def test_ragged_batches(cuda_device, runs, summary, H, D):
    slots, pages = _slots(RUNS[runs], torch.Generator().manual_seed(1))
    _check(cuda_device, slots, pages, H, D, summary=summary)


@pytest.mark.parametrize("H,D", [(1, 8), (3, 40), (8, 128), (2, 256), (5, 64), (7, 264), (1, 512), (2, 576)])
@pytest.mark.parametrize("fused", [0, 1, 3])
def test_heads_and_widths(cuda_device, H, D, fused):
    slots, pages = _slots(RUNS["ragged"], torch.Generator().manual_seed(2))
    _check(cuda_device, slots, pages, H, D, fused=fused, seed=H)


def test_key_and_value_widths_differ_and_padded_cache_rows(cuda_device):
    slots, pages = _slots(RUNS["ragged"], torch.Generator().manual_seed(3))
    _check(cuda_device, slots, pages, 2, 192, Dv=128)
    _check(cuda_device, slots, pages, 2, 64, Dv=136, pad_k=8, pad_v=24, summary=False)
    _check(cuda_device, slots, pages, 2, 128, Dv=128, pad_k=16, pad_v=8)


@pytest.mark.parametrize("summary", [True, False])
def test_latent_rows(cuda_device, summary):
    slots, pages = _slots(RUNS["many"], torch.Generator().manual_seed(4))
    _check(cuda_device, slots, pages, 1, 576, Dv=512, latent=True, summary=summary)


@pytest.mark.parametrize("before", range(16))
def test_long_prompts_at_every_offset(cuda_device, before):
    """Long batches are cut into windows of 16 tokens: runs that begin at each place of a window."""
    slots, pages = _slots([(before, 5200 - before), (0, 30 + before), (before, 5200)], torch.Generator().manual_seed(9))
    _check(cuda_device, slots, pages, 8, 128, seed=before)


def test_a_slot_named_twice_behind_a_full_page(cuda_device):
    """A page's 16 tokens at a window's end, and one of its slots once more behind it."""
    slots, pages = _slots([(0, 5000)], torch.Generator().manual_seed(10))
    slots = slots[:1] + slots[:2031] + [slots[2030]] + slots[2031:]
    _check(cuda_device, slots, pages, 8, 128)


@pytest.mark.parametrize("summary", [True, False])
def test_padding_is_skipped(cuda_device, summary):
    slots, pages = _slots(RUNS["ragged"], torch.Generator().manual_seed(5))
    slots = [-1] + slots[:40] + [-1, -5] + slots[40:] + [-1] * 30
    # Padding cuts a page's tokens into two runs only here, where the second run starts a new page.
    cut = 43
    while cut < len(slots) and slots[cut] % 16 != 0:
        slots[cut] = -1
        cut += 1
    _check(cuda_device, slots, pages, 4, 128, summary=summary)


def test_a_slot_named_twice_keeps_the_later_row(cuda_device):
    _check(cuda_device, [3, 3, 4, 20, 20, 20], 2, 2, 128)
    _check(cuda_device, [16 + i % 5 for i in range(70)], 3, 2, 128)   # a run of more than a page's tokens


def test_slots_of_a_page_in_any_order(cuda_device):
    _check(cuda_device, [7, 3, 0, 12, 33, 32, 47, 18], 3, 4, 128)


@pytest.mark.parametrize("summary", [True, False])
def test_slots_out_of_range(cuda_device, summary):
    _check(cuda_device, [0, 1, 48, 49, 2**31 - 1, 20], 3, 2, 128, summary=summary, err=se.DEVERR_PAGE_RANGE)


def test_matches_the_one_token_append_and_the_rebuild(cuda_device):
    """A prompt stored at once, then one token per request by this call and by the append: same cache."""
    dev = cuda_device
    g = torch.Generator().manual_seed(6)
    H, D, lens = 4, 128, [37, 16, 1, 160]
    slots, pages = _slots([(0, n) for n in lens], g)
    pages += len(lens)
    width = 11
    table = torch.zeros(len(lens), width, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        for j in range(0, n, 16):
            table[b, j // 16] = slots[at + j] // 16
        if n % 16 == 0:
            table[b, n // 16] = pages - len(lens) + b
        at += n
    kn, vn = (_bf16((sum(lens), H, D), g).to(dev) for _ in range(2))
    k1, v1 = (_bf16((len(lens), H, D), g).to(dev) for _ in range(2))
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    table = table.to(dev)
    got = []
    for way in range(2):
        k, v = (torch.zeros(pages, H, 16, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
        s = torch.zeros(pages, H, 2, D, dtype=torch.bfloat16, device=dev)
        kv = se.paged_kv(k, v, s)
        se.se_paged_kv_store(kv, kn, vn, torch.tensor(slots, dtype=torch.int32, device=dev))
        rebuilt = torch.zeros_like(s)
        se.se_quest_build_summaries(se.paged_kv(k, v, rebuilt), table, ln, 16 * width)
        assert torch.equal(rebuilt.view(torch.int16), s.view(torch.int16))
        if way == 0:
            se.se_quest_update_summaries(kv, k1, v1, table, ln)
        else:
            one = [int(table[b, n // 16]) * 16 + n % 16 for b, n in enumerate(lens)]
            se.se_paged_kv_store(kv, k1, v1, torch.tensor(one, dtype=torch.int32, device=dev))
        got.append((k, v, s))
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_empty_batch_and_binding_checks(cuda_device):
    dev = cuda_device
    k = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device=dev)
    kv = se.paged_kv(k, k.clone(), None)
    rows = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=dev)
    slots = lambda n: torch.zeros(n, dtype=torch.int32, device=dev)
    se.se_paged_kv_store(kv, rows(0, 2, 64), rows(0, 2, 64), slots(0))
    for kn, vn, sl, kind in [(rows(3, 2, 64), rows(3, 2, 64), slots(2), ValueError),
                             (rows(3, 2, 64), rows(2, 2, 64), slots(3), ValueError),
                             (rows(3, 1, 64), rows(3, 2, 64), slots(3), ValueError),
                             (rows(3, 2, 64).float(), rows(3, 2, 64), slots(3), TypeError),
                             (rows(3, 2, 64), None, slots(3), se.SparseEngineError),
                             (rows(3, 2, 64).cpu(), rows(3, 2, 64), slots(3), ValueError)]:
        with pytest.raises(kind):
            se.se_paged_kv_store(kv, kn, vn, sl)
    assert int(k.abs().sum()) == 0
