"""Rows quantised into an 8-bit cache and read back, against a run-by-run simulation. Scales are powers of two (or
given), products with them fp32 and one rounding each: every comparison is exact."""
import numpy as np
import pytest
import torch

import oracle.kv8 as k8
import sparse_decode_attention_quest_gb300 as se

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _no_device_errors(se_lib, cuda_device):
    se.se_read_device_error(clear=True)
    yield
    assert se.se_read_device_error(clear=True) == 0


def _slots(runs, g):
    """Slot map of requests holding ``before`` tokens and getting ``new``, pages handed out at random."""
    pages = sum(-(-(b + n) // 16) for b, n in runs)
    perm = torch.randperm(pages, generator=g).tolist()
    slots, at = [], 0
    for b, n in runs:
        slots += [perm[at + (b + i) // 16] * 16 + (b + i) % 16 for i in range(n)]
        at += -(-(b + n) // 16)
    return slots, max(pages, 1)


def _same(got, want):
    """Codes as the values they stand for (-0 and 0 alike are not told apart by value, so by bits but for NaN)."""
    a, b = got.view(torch.uint8).cpu().numpy(), want
    na, nb = np.isnan(k8.VALUES[a]), np.isnan(k8.VALUES[b])
    np.testing.assert_array_equal(na, nb)
    np.testing.assert_array_equal(np.where(na, 0, a), np.where(nb, 0, b))


class Cache:
    def __init__(self, dev, pages, H, D, seed, scales=None):
        g = np.random.default_rng(seed)
        self.codes = {n: g.integers(0, 127, (pages, H, 16, D)).astype(np.uint8) | (g.integers(0, 2, (pages, H, 16, D)) << 7).astype(np.uint8)
                      for n in "kv"}
        e = g.integers(-12, -3, (2, pages, H)) if scales is None else None
        self.scale = {n: (np.exp2(e[i]) if scales is None else scales(g, (pages, H))).astype(np.float32) for i, n in enumerate("kv")}
        self.d = {n: torch.from_numpy(self.codes[n]).to(dev).view(F8) for n in "kv"}
        self.ds = {n: torch.from_numpy(self.scale[n]).to(dev) for n in "kv"}
        self.kv = se.paged_kv8(self.d["k"], self.d["v"], self.ds["k"], self.ds["v"])

    def store(self, kn, vn, slots):
        for n, x in (("k", kn), ("v", vn)):
            k8.store(self.codes[n], self.scale[n], x.double().numpy(), slots)

    def check(self):
        for n in "kv":
            np.testing.assert_array_equal(self.ds[n].cpu().numpy(), self.scale[n])
            _same(self.d[n], self.codes[n])


def _rows(g, T, heads, D, spread=3):
    x = torch.randn(T, heads, D, generator=g) * torch.exp2(torch.randint(-spread, spread + 1, (T, heads, 1), generator=g))
    return x.to(torch.bfloat16)


def _check(dev, slots, pages, H, D, fused=0, seed=0, err=0, change=None, scales=None, stream=None):
    g = torch.Generator().manual_seed(seed)
    c = Cache(dev, pages, H, D, seed, scales)
    kn, vn = (_rows(g, len(slots), fused + H + fused, D) for _ in range(2))
    if change:
        change(kn), change(vn)
    dk, dv = kn.to(dev)[:, fused:fused + H], vn.to(dev)[:, fused:fused + H]
    sm = torch.tensor(slots, dtype=torch.int32, device=dev)
    se.se_paged_kv8_store(c.kv, dk, dv, sm, stream)
    assert se.se_read_device_error(clear=True) == err
    c.store(kn[:, fused:fused + H], vn[:, fused:fused + H], slots)
    c.check()
    se.se_paged_kv8_store(c.kv, dk, dv, sm, stream)   # the same rows again
    assert se.se_read_device_error(clear=True) == err
    c.store(kn[:, fused:fused + H], vn[:, fused:fused + H], slots)
    c.check()


RUNS = {
    "one": [(0, 1)], "one_inside": [(5, 1)], "page": [(0, 16)], "over_a_border": [(9, 13)], "long": [(3, 200)],
    "decode": [(i * 7, 1) for i in range(40)], "ragged": [(0, 33), (15, 1), (16, 1), (31, 66), (7, 9), (0, 1), (48, 16)],
    "many": [(i % 19, 1 + (i * i) % 45) for i in range(90)],
}


@pytest.mark.parametrize("runs", list(RUNS))
@pytest.mark.parametrize("H,D", [(4, 128), (1, 64), (2, 256)])
def test_ragged_batches(cuda_device, runs, H, D):
    slots, pages = _slots(RUNS[runs], torch.Generator().manual_seed(1))
    _check(cuda_device, slots, pages, H, D)


@pytest.mark.parametrize("H", [1, 3, 5, 8, 40])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fused", [0, 3])
def test_heads_and_columns_of_a_wider_tensor(cuda_device, H, D, fused):
    slots, pages = _slots(RUNS["ragged"], torch.Generator().manual_seed(2))
    _check(cuda_device, slots, pages, H, D, fused=fused, seed=H)


@pytest.mark.parametrize("before", [0, 1, 7, 15])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_prompts(cuda_device, before, D):
    """Long batches are cut into windows of 16 tokens: runs that begin at several places of a window."""
    slots, pages = _slots([(before, 5200 - before), (0, 30 + before), (before, 3200)], torch.Generator().manual_seed(9))
    _check(cuda_device, slots, pages, 2, D, seed=before)


def test_padding_and_bad_slots_are_skipped(cuda_device):
    slots, pages = _slots(RUNS["ragged"], torch.Generator().manual_seed(3))
    _check(cuda_device, slots + [-1] * 40, pages, 4, 128)
    assert slots[35] // 16 != slots[36] // 16  # the tokens of a page stand together
    _check(cuda_device, [-1] * 3 + slots[:36] + [-1, -7] + slots[36:], pages, 4, 128)
    _check(cuda_device, slots[:36] + [16 * pages, 2**31 - 1] + slots[36:], pages, 4, 128, err=se.DEVERR_PAGE_RANGE)
    _check(cuda_device, [-1] * 20, 2, 4, 128)


def test_slots_in_any_order_and_named_twice(cuda_device):
    for D in (64, 128, 256):
        _check(cuda_device, [16 * 3 + i for i in (4, 2, 9, 1)] + [16 * 1 + i for i in (15, 0, 7)], 5, 2, D)
        _check(cuda_device, [16 * 3 + i for i in (4, 2, 2, 9)], 5, 2, D)
        _check(cuda_device, [16 * 2 + i % 16 for i in range(40)], 5, 2, D)
        slots, pages = _slots([(0, 4000)], torch.Generator().manual_seed(10))
        _check(cuda_device, slots[:1] + slots[:2031] + [slots[2030]] + slots[2031:], pages, 2, D)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["some", "row", "all"])
def test_values_that_are_not_finite(cuda_device, value, where):
    """They are held as NaN and do not count for the scale."""
    def change(x):
        if where == "some":
            x[::3, :, 5] = value
        elif where == "row":
            x[1::4] = value
        else:
            x.fill_(value)
    for runs in ("ragged", "one_inside", "page"):
        slots, pages = _slots(RUNS[runs], torch.Generator().manual_seed(4))
        _check(cuda_device, slots, pages, 2, 128, change=change)
    _check(cuda_device, [16 * 3 + i for i in (4, 2, 9, 1)], 5, 2, 64, change=change)


@pytest.mark.parametrize("value", [0.0, 1e-39, 2.0 ** -100, 448.0, 449.0, 3.3e38, -3.5, 2.0 ** -91.9])
def test_extreme_values(cuda_device, value):
    def change(x):
        x.mul_(1e-3 * abs(value))
        x[..., 3] = value
    slots, pages = _slots(RUNS["ragged"], torch.Generator().manual_seed(5))
    _check(cuda_device, slots, pages, 2, 128, change=change, scales=lambda g, s: np.full(s, 2.0 ** -100))


@pytest.mark.parametrize("kind", ["odd", "zero", "large"])
def test_scales_that_a_caller_set(cuda_device, kind):
    """A page's present scale need not be a power of two: it is kept, or replaced by a larger one."""
    make = {"odd": lambda g, s: g.uniform(1e-4, 0.1, s), "zero": lambda g, s: np.zeros(s), "large": lambda g, s: np.full(s, 1e20)}[kind]
    slots, pages = _slots(RUNS["many"], torch.Generator().manual_seed(6))
    _check(cuda_device, slots, pages, 2, 128, scales=make)


def test_token_by_token(cuda_device):
    """40 decode steps: scales grow inside pages, and each page ends as the simulation's."""
    dev = cuda_device
    g = torch.Generator().manual_seed(7)
    c = Cache(dev, 12, 3, 128, 7)
    for t in range(40):
        slots = [16 * (t // 16) + t % 16, 16 * (3 + (t + 9) // 16) + (t + 9) % 16, -1]
        kn, vn = _rows(g, 3, 3, 128, 5), _rows(g, 3, 3, 128, 5)
        se.se_paged_kv8_store(c.kv, kn.to(dev), vn.to(dev), torch.tensor(slots, dtype=torch.int32, device=dev))
        c.store(kn, vn, slots)
        c.check()


# ------------------------------------------------------------------ rows back
def _check_load(dev, counts, firsts, H, D, pad=0, fused=0, seed=0, err=0, bad=None, width=None, scales=None, stream=None):
    g = torch.Generator().manual_seed(seed)
    B = len(counts)
    lens = [a + b for a, b in zip(counts, firsts or [0] * B)]
    n = [-(-x // 16) for x in lens]
    pages = max(1, sum(n))
    c = Cache(dev, pages, H, D, seed, scales)
    table = torch.full((B, width or max(n + [1])), -3, dtype=torch.int32)
    perm = torch.randperm(pages, generator=g).int()
    for b in range(B):
        table[b, :n[b]] = perm[sum(n[:b]):sum(n[:b]) + n[b]]
    if bad:
        bad(table)
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    T = int(start[-1]) + pad
    out = [torch.full((T, fused + H + fused, D), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    se.se_paged_kv8_load(c.kv, table.to(dev), torch.from_numpy(start).to(dev), *(o[:, fused:fused + H] for o in out),
                         None if firsts is None else torch.tensor(firsts, dtype=torch.int32, device=dev), stream)
    torch.cuda.synchronize()
    for n_, o in zip("kv", out):
        want, e = k8.load(c.codes[n_], c.scale[n_], table.numpy(), start, np.full((T, H, D), 7.0), firsts)
        assert e == err
        np.testing.assert_array_equal(o[:, fused:fused + H].double().cpu().numpy(), want)
        o[:, fused:fused + H] = 7.0
        assert bool((o == 7.0).all())
    assert se.se_read_device_error(clear=True) == err


@pytest.mark.parametrize("H,D", [(1, 64), (5, 64), (2, 128), (8, 128), (3, 256), (1, 256)])
@pytest.mark.parametrize("fused", [0, 2])
def test_load(cuda_device, H, D, fused):
    _check_load(cuda_device, [33, 0, 1, 16, 0, 0, 250, 7], None, H, D, fused=fused)
    _check_load(cuda_device, [33, 0, 1, 16, 0, 0, 250, 7], [0, 5, 15, 16, 0, 40, 3, 100], H, D, pad=37, fused=fused)


@pytest.mark.parametrize("rows", [1, 2, 15, 64, 65, 4863, 4864, 9728, 20000])
def test_load_of_one_request(cuda_device, rows):
    _check_load(cuda_device, [rows], [9], 1, 64, pad=1, seed=rows)


def test_load_of_many_requests(cuda_device):
    g = np.random.default_rng(3)
    _check_load(cuda_device, g.integers(0, 9, 3000).tolist(), g.integers(0, 30, 3000).tolist(), 1, 64, pad=100)
    _check_load(cuda_device, [0] * 50, None, 2, 128, pad=9)


def test_load_scales_that_are_no_powers_of_two(cuda_device):
    _check_load(cuda_device, [100, 40], None, 2, 128, scales=lambda g, s: g.uniform(1e-4, 0.1, s))


def test_load_reports_and_skips(cuda_device):
    def bad(t):
        t[0, 1], t[1, 0], t[2, 2] = -1, 2**31 - 1, 1000
    _check_load(cuda_device, [40, 16, 60], None, 2, 128, bad=bad, err=se.DEVERR_PAGE_RANGE)
    _check_load(cuda_device, [40, 16, 60], [0, -5, 0], 2, 128, err=se.DEVERR_LENGTH)
    _check_load(cuda_device, [40, 90], None, 2, 128, width=6, err=0)
    dev = cuda_device
    c = Cache(dev, 4, 2, 64, 1)
    out = [torch.full((200, 2, 64), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    table = torch.arange(4, dtype=torch.int32, device=dev).view(1, 4)
    # More rows than the table holds, and more than the outputs hold.
    se.se_paged_kv8_load(c.kv, table, torch.tensor([0, 1000], dtype=torch.int32, device=dev), *out)
    assert se.se_read_device_error(clear=True) == se.DEVERR_LENGTH
    want, _ = k8.load(c.codes["k"], c.scale["k"], table.cpu().numpy(), [0, 200], np.full((200, 2, 64), 7.0))
    np.testing.assert_array_equal(out[0].double().cpu().numpy(), want)


def test_streams(cuda_device):
    s = torch.cuda.Stream(device=cuda_device)
    slots, pages = _slots(RUNS["ragged"], torch.Generator().manual_seed(8))
    _check(cuda_device, slots, pages, 2, 128, stream=s)
    _check_load(cuda_device, [33, 7], None, 2, 128, stream=s)


def test_load_of_the_largest_batch(cuda_device):
    """16,384 requests of up to three rows, a page each."""
    dev, B = cuda_device, 16384
    g = torch.Generator().manual_seed(11)
    counts = torch.randint(0, 4, (B,), generator=g)
    firsts = torch.randint(0, 14, (B,), generator=g)
    c = Cache(dev, B, 1, 64, 11)
    table = torch.randperm(B, generator=g).int()[:, None]
    start = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(counts, 0)]).int()
    T = int(start[-1])
    out = [torch.full((T + 5, 1, 64), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    se.se_paged_kv8_load(c.kv, table.to(dev), start.to(dev), *out, firsts.int().to(dev))
    r = torch.repeat_interleave(torch.arange(B), counts)
    pos = (firsts[r] + torch.arange(T) - start[r]).numpy()
    for n, o in zip("kv", out):
        page = table[r, 0].numpy()
        want = k8.VALUES[c.codes[n][page, :, pos]] * c.scale[n][page].astype(np.float64)[..., None]
        np.testing.assert_array_equal(o[:T].double().cpu().numpy(), want)
        assert bool((o[T:] == 7.0).all())
    with pytest.raises(se.SparseEngineError, match="batch >"):
        z = torch.zeros(B + 2, dtype=torch.int32, device=dev)
        se.se_paged_kv8_load(c.kv, torch.zeros(B + 1, 1, dtype=torch.int32, device=dev), z, *out)


def test_recorded_store_and_load(cuda_device):
    """Recorded once; the replays take the slots, rows and spans that their buffers hold then."""
    dev = cuda_device
    s = torch.cuda.Stream(device=dev)
    c = Cache(dev, 6, 2, 128, 12)
    kn, vn = (torch.zeros(20, 2, 128, dtype=torch.bfloat16, device=dev) for _ in range(2))
    slots = torch.full((20,), -1, dtype=torch.int32, device=dev)
    table = torch.arange(6, dtype=torch.int32, device=dev).view(2, 3)
    start = torch.zeros(3, dtype=torch.int32, device=dev)
    out = [torch.zeros(96, 2, 128, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    torch.cuda.synchronize()
    se.se_capture_begin(s)
    se.se_paged_kv8_store(c.kv, kn, vn, slots, s)
    se.se_paged_kv8_load(c.kv, table, start, *out, stream=s)
    step = se.se_capture_end(s)
    g = torch.Generator().manual_seed(13)
    for i, (a, b) in enumerate([(20, 0), (7, 13), (0, 16)]):
        new = [_rows(g, 20, 2, 128) for _ in range(2)]
        at = [16 * (i % 2) + j for j in range(a)] + [48 + 16 * i + j for j in range(b)] + [-1] * (20 - a - b)
        slots.copy_(torch.tensor(at, dtype=torch.int32))
        kn.copy_(new[0])
        vn.copy_(new[1])
        start.copy_(torch.tensor([0, 30 + i, 70], dtype=torch.int32))
        for o in out:
            o.fill_(7.0)
        torch.cuda.synchronize()
        step.launch(s)
        s.synchronize()
        c.store(*new, at)
        c.check()
        for n, o in zip("kv", out):
            want, err = k8.load(c.codes[n], c.scale[n], table.cpu().numpy(), [0, 30 + i, 70], np.full(o.shape, 7.0))
            assert err == 0
            np.testing.assert_array_equal(o.double().cpu().numpy(), want)
