"""Dense paged decode on the GPU against the fp64 oracle.

Error bounds, from the arithmetic: the kernel's logits are fp32 sums of exact products of bf16
values (each of the D additions off by at most 2^-23 of the running magnitude, truncation allowed
for), scaled once; exp2 is good to 2^-22; a probability is rounded to bf16 (half a step, 2^-8 of its
value) before it meets its value row, while l sums the unrounded ones; every other sum and the
merge of splits are fp32; the output is rounded to bf16 once. With dz = (D + 8) 2^-23 max_j sum_c
|s q_c k_jc| and A = sum_j alpha_j |v_j|,
    |out - exact| <= (2^-8 + 2 dz + (n + 64) 2^-23) A + 2^-8 |exact| (1 + 2^-7) + 2^-133,
    |lse - exact| <= dz + (n + 64) 2^-23 + 2^-21 (1 + |exact|).
"""
import math

import numpy as np
import pytest
import torch

import oracle.paged as op
import sparse_decode_attention_quest_gb300 as se

pytestmark = pytest.mark.gpu

GUARD = 77.0


@pytest.fixture(autouse=True)
def _no_device_errors(se_lib, cuda_device):
    se.se_read_device_error(clear=True)
    yield
    assert se.se_read_device_error(clear=True) == 0


class Inputs:
    """A paged cache whose unkept rows hold NaN and infinities, on the CPU and on the GPU."""

    def __init__(self, dev, lens, Hq, H, D, latent=False, seed=0, pad=0, q_pad=0, sink=0, recent=0, extra_pages=3,
                 scale=None, key_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hq, self.H, self.D = lens, Hq, H, D
        self.Dv = 512 if latent else D
        self.sink, self.recent, self.dev = sink, recent, dev
        self.scale = 1.0 / math.sqrt(D) if scale is None else scale
        n = [-(-x // 16) for x in lens]
        total = sum(n) + extra_pages
        perm = torch.randperm(total, generator=g)
        width = max(n + [1]) + 1
        self.table = torch.full((len(lens), width), -5, dtype=torch.int32)  # behind a request's pages: never read
        at = 0
        for b, m in enumerate(n):
            self.table[b, :m] = perm[at:at + m].int()
            at += m
        self.k = (torch.randn(total, H, 16, D + pad, generator=g) * key_scale).to(torch.bfloat16)
        self.v = None if latent else torch.randn(total, H, 16, D + pad, generator=g).to(torch.bfloat16)
        junk = torch.tensor([float("nan"), float("inf"), -float("inf")], dtype=torch.bfloat16)
        kept = torch.zeros(total, 16, dtype=torch.bool)
        for b, L in enumerate(lens):
            j = torch.from_numpy(op.kept_positions(L, sink, recent)).long()
            kept[self.table[b, j // 16].long(), j % 16] = True
        drop = (~kept).nonzero()
        for t in (self.k, self.v):
            if t is not None:
                t[drop[:, 0], :, drop[:, 1]] = junk[torch.arange(len(drop)) % 3][:, None, None]
        self.q_all = torch.randn(len(lens), Hq + q_pad, D, generator=g).to(torch.bfloat16)
        self.q = self.q_all[:, :Hq]
        self.dk, self.dv = self.k.to(dev), None if self.v is None else self.v.to(dev)
        self.kv = se.paged_kv(self.dk, self.dv, None, self.Dv)
        self.kv.head_dim, self.kv.head_dim_v = D, self.Dv
        self.dq = self.q_all.to(dev)[:, :Hq]
        self.dt = self.table.to(dev)
        self.dl = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.ws = torch.zeros(se.se_paged_decode_workspace_size(len(lens), Hq, H, D, self.Dv), dtype=torch.uint8,
                              device=dev)

    def run(self, lse=True, ws=None, stream=None):
        B = len(self.lens)
        out = torch.full((B + 1, self.Hq, self.Dv), GUARD, dtype=torch.bfloat16, device=self.dev)
        ls = torch.full((B + 1, self.Hq), GUARD, dtype=torch.float32, device=self.dev)
        se.se_paged_decode(self.kv, self.dq, self.dt, self.dl, self.scale, out[:B], ls[:B] if lse else None,
                           self.ws if ws is None else ws, self.sink, self.recent, stream)
        torch.cuda.synchronize()
        assert bool((out[B] == GUARD).all()) and bool((ls[B:] == GUARD).all())  # rows behind the batch
        assert not bool((self.ws if ws is None else ws)[:768].any())            # the counters are back at zero
        return out[:B], ls[:B] if lse else None

    def oracle(self):
        v = None if self.v is None else self.v[..., :self.D].float().numpy()
        return op.decode(self.k[..., :self.D].float().numpy(), v, self.table.numpy(), self.lens,
                         self.q.float().numpy(), self.scale, self.Dv, self.sink, self.recent)

    def check(self):
        out, lse = self.run()
        ref, rlse, mag, zmag = self.oracle()
        n = np.array([len(op.kept_positions(L, self.sink, self.recent)) for L in self.lens])[:, None]
        dz = (self.D + 8) * 2.0 ** -23 * zmag
        tol = (2.0 ** -8 + 2 * dz + (n + 64) * 2.0 ** -23)[..., None] * mag + 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7)
        err = np.abs(out.double().cpu().numpy() - ref)
        assert np.isfinite(err).all()
        worst = (err - tol - 2.0 ** -133).max() if err.size else 0.0
        assert worst <= 0, f"out off by {err.max():.3g}, {worst:.3g} beyond its bound"
        got = lse.double().cpu().numpy()
        empty = np.isneginf(rlse)
        assert (np.isneginf(got) == empty).all()
        ltol = dz + (n + 64) * 2.0 ** -23 + 2.0 ** -21 * (1 + np.abs(np.where(empty, 0, rlse)))
        lerr = np.abs(np.where(empty, 0, got) - np.where(empty, 0, rlse))
        assert (lerr <= ltol).all(), f"lse off by {lerr.max():.3g}"
        again, alse = self.run()
        assert torch.equal(again.view(torch.int16), out.view(torch.int16)) and torch.equal(alse, lse)
        return out, lse


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 257, 700]


@pytest.mark.parametrize("Hq,H,D", [(4, 1, 128), (8, 8, 128), (32, 8, 128), (12, 4, 64), (8, 1, 256)])
def test_edge_lengths(cuda_device, Hq, H, D):
    Inputs(cuda_device, EDGES, Hq, H, D, seed=1).check()


@pytest.mark.parametrize("Hq,H", [(1, 1), (5, 1), (8, 1), (9, 1), (16, 1), (17, 1), (32, 1), (47, 1), (64, 1), (33, 3),
                                  (14, 2), (3, 3), (10, 5), (6, 6), (28, 4), (7, 7), (40, 8), (18, 9), (10, 10),
                                  (11, 11), (26, 13), (32, 16), (128, 2), (27, 3)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_head_layouts(cuda_device, Hq, H, D):
    Inputs(cuda_device, [70, 0, 333, 1], Hq, H, D, seed=Hq).check()


@pytest.mark.parametrize("Hq", [16, 32, 48, 64])
def test_latent_head_counts(cuda_device, Hq):
    Inputs(cuda_device, [70, 0, 1030, 1, 64, 65], Hq, 1, 576, latent=True, seed=Hq).check()


def test_latent_edge_lengths(cuda_device):
    Inputs(cuda_device, EDGES, 64, 1, 576, latent=True, seed=2).check()


WINDOWS = [(0, 1), (0, 16), (0, 100), (1, 1), (4, 60), (16, 16), (17, 15), (64, 200), (40, 3), (300, 7), (5, 100000)]


@pytest.mark.parametrize("sink,recent", WINDOWS)
@pytest.mark.parametrize("shape", [(8, 2, 128), (12, 4, 64), (6, 1, 256), (32, 1, 576)])
def test_windows(cuda_device, sink, recent, shape):
    Hq, H, D = shape
    Inputs(cuda_device, [0, 1, 5, 16, 17, 40, 41, 99, 320, 333, 1000], Hq, H, D, latent=D == 576, sink=sink,
           recent=recent, seed=3).check()


@pytest.mark.parametrize("batch,lo,hi", [(1, 20011, 20011), (5, 0, 3000), (150, 1, 70)])
@pytest.mark.parametrize("shape", [(16, 1, 128), (36, 3, 128), (34, 2, 128), (32, 2, 64), (30, 1, 256), (40, 1, 256)])
def test_many_heads_over_split_items(cuda_device, batch, lo, hi, shape):
    """Tiles of eight and of sixteen query heads, alone in their warp and sharing pages, whole and joined."""
    g = torch.Generator().manual_seed(batch + hi)
    lens = torch.randint(lo, hi + 1, (batch,), generator=g).tolist()
    Inputs(cuda_device, lens, *shape, seed=batch).check()


@pytest.mark.parametrize("Hq,H,D", [(1000, 1000, 64), (130, 65, 128)])
def test_many_kv_heads(cuda_device, Hq, H, D):
    """More (request, head group) items than CTAs from few requests, and about as many."""
    Inputs(cuda_device, [100, 0, 17], Hq, H, D, seed=H).check()
    Inputs(cuda_device, [33], Hq, H, D, seed=H).check()


@pytest.mark.parametrize("batch", [19, 76, 151, 152, 153, 160, 161])
@pytest.mark.parametrize("shape", [(8, 2, 128), (9, 3, 64), (8, 8, 128), (12, 1, 256), (16, 1, 576)])
def test_about_one_short_request_per_cta(cuda_device, batch, shape):
    """Around the batch sizes at which every piece of a request still gets a CTA of its own."""
    Hq, H, D = shape
    lens = [(0, 1, 64, 65, 128, 129, 16, 200, 0, 33, 7)[(b * b + b // 5) % 11] for b in range(batch)]
    Inputs(cuda_device, lens, Hq, H, D, latent=D == 576, seed=batch).check()
    Inputs(cuda_device, [100] * batch, Hq, H, D, latent=D == 576, seed=batch, sink=4, recent=70).check()


@pytest.mark.parametrize("batch,lo,hi", [(1, 4096, 4096), (1, 20011, 20011), (3, 1, 9000), (70, 0, 400), (300, 0, 64),
                                         (51, 208, 208), (160, 330, 350), (200, 1, 17), (33, 1500, 1600), (2, 1, 30000)])
@pytest.mark.parametrize("shape", [(8, 2, 128), (4, 1, 64), (16, 8, 64), (2, 1, 256), (64, 1, 576)])
def test_splits(cuda_device, batch, lo, hi, shape):
    """Few long requests over many CTAs, many short ones in one, and ragged mixes."""
    Hq, H, D = shape
    g = np.random.default_rng(batch)
    if D == 576:
        batch, hi = min(batch, 120), min(hi, 20011)
        lo = min(lo, hi)
    Inputs(cuda_device, g.integers(lo, hi + 1, batch).tolist(), Hq, H, D, latent=D == 576, seed=4).check()


@pytest.mark.parametrize("pad,q_pad", [(8, 0), (64, 0), (0, 3), (24, 9)])
@pytest.mark.parametrize("shape", [(8, 2, 128), (4, 1, 64), (6, 3, 256), (16, 1, 576)])
def test_strides(cuda_device, pad, q_pad, shape):
    """Cache rows further apart than their width, queries as columns of a wider tensor."""
    Hq, H, D = shape
    Inputs(cuda_device, [70, 333, 17], Hq, H, D, latent=D == 576, pad=pad, q_pad=q_pad, seed=5).check()


@pytest.mark.parametrize("shape", [(8, 2, 128), (64, 1, 576)])
@pytest.mark.parametrize("scale", [0.0, -0.07, 1.0])
def test_scales(cuda_device, shape, scale):
    Hq, H, D = shape
    Inputs(cuda_device, [70, 333, 17], Hq, H, D, latent=D == 576, scale=scale, seed=6, key_scale=0.5).check()


def test_rising_logits_move_the_maximum(cuda_device):
    """Every later page beats all before it: the running maximum moves at each."""
    for shape in [(8, 2, 128), (32, 1, 576)]:
        Hq, H, D = shape
        x = Inputs(cuda_device, [1500], Hq, H, D, latent=D == 576, seed=7)
        j = torch.arange(1500)
        ramp = (j.float() / 100)[:, None, None]
        q0 = x.q[0].float().mean(0) / 4
        rows = (x.k[x.table[0, j // 16].long(), :, j % 16][..., :D].float() * 0.1 + ramp * q0).to(torch.bfloat16)
        x.k[x.table[0, j // 16].long(), :, j % 16] = rows
        x.dk.copy_(x.k)
        x.check()


@pytest.mark.parametrize("D", [128, 576])
def test_infinite_logits(cuda_device, D):
    """Keys that make logits -inf carry no weight; a row of nothing else is empty."""
    dev = cuda_device
    Hq, H = (8, 2) if D == 128 else (16, 1)
    x = Inputs(dev, [40, 20, 33], Hq, H, D, latent=D == 576, seed=8)
    x.q_all[:, :, 0] = 1.0
    x.dq.copy_(x.q)
    neg = [(0, j) for j in range(0, 20)] + [(1, j) for j in range(20)] + [(2, 32)]
    for b, j in neg:
        x.k[x.table[b, j // 16].long(), :, j % 16, D - 1 if D == 576 else 0] = -float("inf")
    if D == 576:
        x.q_all[:, :, D - 1] = 1.0
        x.dq.copy_(x.q)
    x.dk.copy_(x.k)
    out, lse = x.run()
    kept = {0: range(20, 40), 1: range(0), 2: range(32)}
    for b, js in kept.items():
        if not len(js):
            assert bool((out[b] == 0).all()) and bool(torch.isneginf(lse[b]).all())
            continue
        js = torch.tensor(list(js))
        for a in range(Hq):
            h = a // (Hq // H)
            keys = x.k[x.table[b, js // 16].long(), h, js % 16].double()
            vals = keys[:, :512] if D == 576 else x.v[x.table[b, js // 16].long(), h, js % 16].double()
            z = x.scale * (keys @ x.q[b, a].double())
            ref = torch.softmax(z, 0) @ vals
            mag = torch.softmax(z, 0) @ vals.abs()
            tol = (2.0 ** -8 + 1e-4) * mag + 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -7)
            assert bool(((out[b, a].double().cpu() - ref).abs() <= tol).all())
            assert abs(float(lse[b, a]) - float(torch.logsumexp(z, 0))) < 1e-4


def test_nan_in_a_kept_value_stays_in_its_column(cuda_device):
    x = Inputs(cuda_device, [50, 50], 8, 2, 128, seed=9)
    x.v[x.table[0, 1].long(), 1, 4, 7] = float("nan")
    x.dv.copy_(x.v)
    out, _ = x.run()
    bad = torch.isnan(out).cpu()
    want = torch.zeros_like(bad)
    want[0, 4:8, 7] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("shape", [(8, 2, 128), (16, 1, 576)])
def test_no_lse(cuda_device, shape):
    Hq, H, D = shape
    x = Inputs(cuda_device, [70, 0, 333], Hq, H, D, latent=D == 576, seed=10)
    a, _ = x.run()
    b, _ = x.run(lse=False)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("shape", [(8, 2, 128), (16, 1, 576)])
def test_one_workspace_for_other_lengths_and_streams(cuda_device, shape):
    """Calls in a row share a workspace; the second runs on another stream, behind an event."""
    Hq, H, D = shape
    x = Inputs(cuda_device, [5000, 3], Hq, H, D, latent=D == 576, seed=11)
    want, _ = x.run()
    y = Inputs(cuda_device, [7, 2500], Hq, H, D, latent=D == 576, seed=12)
    y.check()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            y.run(ws=x.ws)
        got, _ = x.run(ws=x.ws, stream=s)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("shape", [(8, 2, 128), (16, 1, 576)])
def test_bad_pages_and_lengths_are_reported_and_skipped(cuda_device, shape):
    Hq, H, D = shape
    lat = D == 576
    x = Inputs(cuda_device, [64, 40, 33, 16], Hq, H, D, latent=lat, seed=13)
    for bad in (-1, x.k.shape[0], 2**31 - 1):
        x.dt[0, 1] = bad
        out, lse = x.run()
        assert se.se_read_device_error(clear=True) == se.DEVERR_PAGE_RANGE
        # Request 0 without its second page: as if its first, third and fourth were all it had.
        y = Inputs(cuda_device, [48, 40, 33, 16], Hq, H, D, latent=lat, seed=13)
        y.k, y.v, y.dk, y.dv, y.kv = x.k, x.v, x.dk, x.dv, x.kv
        y.table, y.dt = x.table.clone(), x.table.clone().to(cuda_device)
        y.table[0, 1:3] = x.table[0, 2:4]
        y.dt[0, 1:3] = y.dt[0, 2:4].clone()
        y.q, y.dq = x.q, x.dq
        ref, rlse, mag, _ = y.oracle()
        assert (np.abs(out.double().cpu().numpy() - ref) <= 2.0 ** -7 * (mag + np.abs(ref)) + 1e-5).all()
        assert np.abs(lse.cpu().numpy() - rlse).max() < 1e-4
    x.dt.copy_(x.table)
    good, _ = x.run()
    x.dl[2] = -4
    out, lse = x.run()
    assert se.se_read_device_error(clear=True) == se.DEVERR_LENGTH
    assert bool((out[2] == 0).all()) and bool(torch.isneginf(lse[2]).all())
    assert torch.equal(out[0].view(torch.int16), good[0].view(torch.int16))
    x.dl[2] = 16 * x.dt.shape[1] + 1  # longer than its table: clipped; the table's end is out of range too
    x.run()
    assert se.se_read_device_error(clear=True) == se.DEVERR_LENGTH | se.DEVERR_PAGE_RANGE


def test_agrees_with_the_sparse_decode_over_every_page(cuda_device):
    """The selected-pages decode told to take every page gives the same attention."""
    dev = cuda_device
    x = Inputs(dev, [4096, 700, 33], 32, 4, 128, seed=14)
    n = [-(-L // 16) for L in x.lens]
    sel = torch.zeros(3, 4, max(n), dtype=torch.int32, device=dev)
    cnt = torch.zeros(3, 4, dtype=torch.int32, device=dev)
    for b, m in enumerate(n):
        sel[b, :, :m] = torch.arange(m, device=dev)
        cnt[b] = m
    out = torch.empty(3, 32, 128, dtype=torch.bfloat16, device=dev)
    lse = torch.empty(3, 32, device=dev)
    ws = torch.zeros(se.se_sparse_decode_workspace_size(3, 32, 4, 128, max(n)), dtype=torch.uint8, device=dev)
    kv = se.paged_kv(x.dk, x.dv, None)
    se.se_sparse_paged_decode(kv, x.dq.contiguous(), x.dt, x.dl, sel, cnt, x.scale, out, lse, ws)
    mine, mlse = x.run()
    ref, rlse, mag, _ = x.oracle()
    assert float((mlse - lse).abs().max()) < 1e-4
    assert (np.abs((mine.double() - out.double()).cpu().numpy()) <= 2.0 ** -6 * (mag + np.abs(ref))).all()


@pytest.mark.parametrize("batch,shape", [(4096, (2, 1, 64)), (512, (16, 1, 576))])
def test_largest_batches(cuda_device, batch, shape):
    Hq, H, D = shape
    g = np.random.default_rng(1)
    Inputs(cuda_device, g.integers(0, 24, batch).tolist(), Hq, H, D, latent=D == 576, seed=16).check()
    with pytest.raises(se.SparseEngineError, match="batch >"):
        z = lambda *n: torch.zeros(*n, dtype=torch.int32, device=cuda_device)
        bf = lambda *n: torch.zeros(*n, dtype=torch.bfloat16, device=cuda_device)
        k = bf(1, H, 16, D)
        dv = 512 if D == 576 else D
        se.se_paged_decode(se.paged_kv(k, None if D == 576 else k.clone(), None, dv), bf(batch + 1, Hq, D),
                           z(batch + 1, 1), z(batch + 1), 0.1, bf(batch + 1, Hq, dv), None,
                           torch.zeros(64 << 20, dtype=torch.uint8, device=cuda_device))


@pytest.mark.parametrize("H,D,pages", [(8, 128, 140000), (1, 576, 240000)])
def test_a_cache_of_more_than_two_to_the_31_elements(cuda_device, H, D, pages):
    """Rows written to and read from the pages at both ends of a 4.5 GB cache."""
    dev = cuda_device
    latent = D == 576
    Hq, dv = (16, 512) if latent else (8, 128)
    assert pages * H * 16 * D > 2 ** 31
    g = torch.Generator().manual_seed(17)
    k = torch.empty(pages, H, 16, D, dtype=torch.bfloat16, device=dev)
    v = None if latent else torch.empty_like(k)
    n = [300, 77]
    ids = [[pages - 1 - i for i in range(19)], [0, pages - 20, 1, pages // 2, pages - 21]]
    table = torch.zeros(2, 19, dtype=torch.int32)
    for b in range(2):
        table[b, :len(ids[b])] = torch.tensor(ids[b], dtype=torch.int32)
    slots = torch.tensor([ids[b][j // 16] * 16 + j % 16 for b in range(2) for j in range(n[b])], dtype=torch.int32)
    kn = torch.randn(sum(n), H, D, generator=g).to(torch.bfloat16)
    vn = None if latent else torch.randn(sum(n), H, D, generator=g).to(torch.bfloat16)
    kv = se.paged_kv(k, v, None, dv)
    se.se_paged_kv_store(kv, kn.to(dev), None if latent else vn.to(dev), slots.to(dev))
    q = torch.randn(2, Hq, D, generator=g).to(torch.bfloat16)
    out = torch.empty(2, Hq, dv, dtype=torch.bfloat16, device=dev)
    lse = torch.empty(2, Hq, device=dev)
    ws = torch.zeros(se.se_paged_decode_workspace_size(2, Hq, H, D, dv), dtype=torch.uint8, device=dev)
    scale = 1.0 / math.sqrt(D)
    se.se_paged_decode(kv, q.to(dev), table.to(dev), torch.tensor(n, dtype=torch.int32, device=dev), scale, out, lse, ws)
    # The same rows in a small cache, for the oracle.
    m = -(-sum(n) // 16) + 2
    small_k, small_v = np.zeros((m, H, 16, D)), None if latent else np.zeros((m, H, 16, D))
    st = np.zeros((2, 19), dtype=np.int64)
    at = 0
    for b in range(2):
        st[b, :len(ids[b])] = np.arange(len(ids[b])) + at
        for j in range(n[b]):
            row = sum(n[:b]) + j
            small_k[st[b, j // 16], :, j % 16] = kn[row].float().numpy()
            if not latent:
                small_v[st[b, j // 16], :, j % 16] = vn[row].float().numpy()
        at += len(ids[b])
    ref, rlse, mag, _ = op.decode(small_k, small_v, st, n, q.float().numpy(), scale, dv)
    tol = (2.0 ** -8 + 1e-4) * mag + 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7)
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    assert np.abs(lse.cpu().numpy() - rlse).max() < 1e-4


def test_binding_checks(cuda_device):
    x = Inputs(cuda_device, [5, 6], 8, 2, 128, seed=15)
    out = torch.empty(2, 8, 128, dtype=torch.bfloat16, device=cuda_device)
    lse = torch.empty(2, 8, device=cuda_device)
    good = dict(kv=x.kv, q=x.dq, block_table=x.dt, seq_lens=x.dl, sm_scale=0.1, out=out, out_lse=lse, workspace=x.ws)
    se.se_paged_decode(**good)
    for name, bad, kind in [("q", x.dq[0], ValueError), ("q", x.dq.float(), TypeError), ("q", x.q, ValueError),
                            ("q", x.dq[:, :, :64], ValueError), ("block_table", x.dt[:1], ValueError),
                            ("seq_lens", x.dl[:1], ValueError), ("seq_lens", x.dl.long(), TypeError),
                            ("out", out[:1], ValueError), ("out", out.float(), TypeError), ("out_lse", lse[:1], ValueError),
                            ("out_lse", lse.half(), TypeError), ("workspace", x.ws[:8], se.SparseEngineError),
                            ("workspace", None, se.SparseEngineError), ("sm_scale", float("nan"), se.SparseEngineError)]:
        with pytest.raises(kind):
            se.se_paged_decode(**{**good, name: bad})
    with pytest.raises(se.SparseEngineError, match="sink_tokens without"):
        se.se_paged_decode(**good, sink_tokens=4)
