"""Decode over an 8-bit cache on the GPU against the fp64 oracle over the values that its codes stand for.

Error bounds, from the arithmetic. A query row is scaled by a power of two to a largest magnitude M of 224 to 448 and
enters as fp16, exact or within 2^-25: 2^-32 of M. Its products with codes are exact and summed in fp32 (each of
the D additions off by at most 2^-23 of the running magnitude, truncation allowed for), then scaled in three
multiplications; exp2 is good to 2^-22; a weight meets its value row as fp16 (half a step, 2^-11 of it, or 2^-25 where the largest
product of weight and V scale is 2^14 at least: 2^-39 of that, S, against codes up to 448) while l sums the unrounded ones;
its exponent, up to 2^7 where the scales of pages differ widely, is rounded by 2^-18 (2^-17 of the weight, which the n + 64
roundings below are 2^-17 or more for); every other sum and the merge of splits are fp32; the output is rounded to bf16 once.
With dz = |s| (2^-32 M max_j sum_c |k_jc| + (D + 12) 2^-23 max_j sum_c |q_c k_jc|) and A = sum_j alpha_j |v_j|,
    |out - exact| <= (2^-11 + 2 dz + (n + 64) 2^-23) A + n 2^-39 448 S + 2^-8 |exact| (1 + 2^-7) + 2^-133,
    |lse - exact| <= dz + (n + 64) 2^-23 + 2^-21 (1 + |exact|).
"""
import math

import numpy as np
import pytest
import torch

import oracle.kv8 as k8
import oracle.paged as op
import sparse_decode_attention_quest_gb300 as se

pytestmark = pytest.mark.gpu

GUARD = 77.0
F8 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _no_device_errors(se_lib, cuda_device):
    se.se_read_device_error(clear=True)
    yield
    assert se.se_read_device_error(clear=True) == 0


class Inputs:
    """An 8-bit cache whose unkept rows hold NaN codes, on the CPU and on the GPU."""

    def __init__(self, dev, lens, Hq, H, D, seed=0, q_pad=0, sink=0, recent=0, extra_pages=3, scale=None, spread=2,
                 odd_scales=False, q_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hq, self.H, self.D = lens, Hq, H, D
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
        kept = torch.zeros(total, 16, dtype=torch.bool)
        for b, L in enumerate(lens):
            j = torch.from_numpy(op.kept_positions(L, sink, recent)).long()
            kept[self.table[b, j // 16].long(), j % 16] = True
        self.codes, self.s = {}, {}
        for name in "kv":
            s = torch.exp2(torch.randint(-7 - spread, -7 + spread + 1, (total, H), generator=g).float())
            if odd_scales:
                s = s * (0.6 + torch.rand(total, H, generator=g))
            x = torch.randn(total, H, 16, D, generator=g) * 100  # codes use the range up to 448
            c = x.clamp(-448, 448).to(F8).view(torch.uint8).clone()
            drop = (~kept).nonzero()
            c[drop[:, 0], :, drop[:, 1]] = 0x7F
            # Pages without a kept token: their scales are not used.
            s[~kept.any(1)] = float("nan")
            self.codes[name], self.s[name] = c, s
        self.q_all = (torch.randn(len(lens), Hq + q_pad, D, generator=g) * q_scale).to(torch.bfloat16)
        self.q = self.q_all[:, :Hq]
        self.dt = self.table.to(dev)
        self.dl = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.ws = torch.zeros(se.se_paged_kv8_decode_workspace_size(len(lens), Hq, H, D), dtype=torch.uint8, device=dev)
        self.upload()

    def upload(self):
        self.d = {n: c.to(self.dev).view(F8) for n, c in self.codes.items()}
        self.ds = {n: s.to(self.dev) for n, s in self.s.items()}
        self.kv = se.paged_kv8(self.d["k"], self.d["v"], self.ds["k"], self.ds["v"])
        self.dq = self.q_all.to(self.dev)[:, :self.Hq]

    def value(self, name):
        return k8.values(self.codes[name].numpy(), self.s[name].numpy())

    def run(self, lse=True, ws=None, stream=None):
        B = len(self.lens)
        out = torch.full((B + 1, self.Hq, self.D), GUARD, dtype=torch.bfloat16, device=self.dev)
        ls = torch.full((B + 1, self.Hq), GUARD, dtype=torch.float32, device=self.dev)
        torch.cuda.synchronize()
        se.se_paged_kv8_decode(self.kv, self.dq, self.dt, self.dl, self.scale, out[:B], ls[:B] if lse else None,
                               self.ws if ws is None else ws, self.sink, self.recent, stream)
        torch.cuda.synchronize()
        assert bool((out[B] == GUARD).all()) and bool((ls[B:] == GUARD).all())  # rows behind the batch
        assert not bool((self.ws if ws is None else ws)[:768].any())            # the counters are back at zero
        return out[:B], ls[:B] if lse else None

    def bounds(self):
        """(exact output, log-sum-exp, their bounds)."""
        k, v, q = self.value("k"), self.value("v"), self.q.double().numpy()
        ref, rlse, mag, zmag = op.decode(k, v, self.table.numpy(), self.lens, q, self.scale, self.D, self.sink, self.recent)
        B, G = len(self.lens), self.Hq // self.H
        kmag, top = np.zeros((B, self.Hq)), np.zeros((B, self.Hq))  # top: the largest product of weight and V scale
        for b, L in enumerate(self.lens):
            j = op.kept_positions(L, self.sink, self.recent)
            if len(j):
                page = self.table.numpy()[b, j // 16]
                kmag[b] = np.repeat(np.abs(k[page, :, j % 16]).sum(2).max(0), G)
                z = self.scale * np.einsum("agd,nad->nag", q[b].reshape(self.H, G, -1), k[page, :, j % 16])
                w = np.exp(z - np.where(np.isneginf(rlse[b]), 0, rlse[b]).reshape(self.H, G))
                top[b] = (w * self.s["v"].numpy()[page][:, :, None]).max(0).reshape(-1)
        n = np.array([len(op.kept_positions(L, self.sink, self.recent)) for L in self.lens])[:, None]
        dz = abs(self.scale) * 2.0 ** -32 * np.abs(q).max(2) * kmag + (self.D + 12) * 2.0 ** -23 * zmag
        tol = (2.0 ** -11 + 2 * dz + (n + 64) * 2.0 ** -23)[..., None] * mag + (n * 2.0 ** -39 * 448 * top)[..., None]
        tol = tol + 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7) + 2.0 ** -133
        ltol = dz + (n + 64) * 2.0 ** -23 + 2.0 ** -21 * (1 + np.abs(np.where(np.isneginf(rlse), 0, rlse)))
        return ref, rlse, tol, ltol

    def check(self):
        out, lse = self.run()
        ref, rlse, tol, ltol = self.bounds()
        err = np.abs(out.double().cpu().numpy() - ref)
        assert np.isfinite(err).all()
        worst = (err - tol).max() if err.size else 0.0
        assert worst <= 0, f"out off by {err.max():.3g}, {worst:.3g} beyond its bound"
        got = lse.double().cpu().numpy()
        empty = np.isneginf(rlse)
        assert (np.isneginf(got) == empty).all()
        lerr = np.abs(np.where(empty, 0, got) - np.where(empty, 0, rlse))
        assert (lerr <= ltol).all(), f"lse off by {lerr.max():.3g}"
        again, alse = self.run()
        assert torch.equal(again.view(torch.int16), out.view(torch.int16)) and torch.equal(alse, lse)
        return out, lse


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 257, 700]
SHAPES = [(8, 2, 128), (12, 4, 64), (6, 1, 256)]


@pytest.mark.parametrize("Hq,H,D", [(4, 1, 128), (8, 8, 128), (32, 8, 128), (12, 4, 64), (8, 1, 256), (4, 1, 64)])
def test_edge_lengths(cuda_device, Hq, H, D):
    Inputs(cuda_device, EDGES, Hq, H, D, seed=1).check()


@pytest.mark.parametrize("Hq,H", [(1, 1), (5, 1), (8, 1), (9, 1), (16, 1), (17, 1), (32, 1), (47, 1), (64, 1), (33, 3),
                                  (14, 2), (3, 3), (10, 5), (6, 6), (28, 4), (7, 7), (40, 8), (18, 9), (10, 10),
                                  (11, 11), (26, 13), (32, 16), (128, 2), (27, 3)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_head_layouts(cuda_device, Hq, H, D):
    Inputs(cuda_device, [70, 0, 333, 1], Hq, H, D, seed=Hq).check()


WINDOWS = [(0, 1), (0, 16), (0, 100), (1, 1), (4, 60), (16, 16), (17, 15), (64, 200), (40, 3), (300, 7), (5, 100000)]


@pytest.mark.parametrize("sink,recent", WINDOWS)
@pytest.mark.parametrize("shape", SHAPES)
def test_windows(cuda_device, sink, recent, shape):
    Inputs(cuda_device, [0, 1, 5, 16, 17, 40, 41, 99, 320, 333, 1000], *shape, sink=sink, recent=recent, seed=3).check()


@pytest.mark.parametrize("batch,lo,hi", [(1, 4096, 4096), (1, 20011, 20011), (3, 1, 9000), (70, 0, 400), (300, 0, 64),
                                         (160, 330, 350), (200, 1, 17), (33, 1500, 1600), (2, 1, 30000)])
@pytest.mark.parametrize("shape", [(8, 2, 128), (4, 1, 64), (16, 8, 64), (2, 1, 256), (32, 1, 128), (18, 1, 256)])
def test_splits(cuda_device, batch, lo, hi, shape):
    """Few long requests over many CTAs, many short ones in one, and ragged mixes."""
    g = np.random.default_rng(batch)
    Inputs(cuda_device, g.integers(lo, hi + 1, batch).tolist(), *shape, seed=4).check()


@pytest.mark.parametrize("lens,sink,recent", [([20011], 0, 0), ([9000, 1, 0, 4095], 0, 0), ([330] * 160, 0, 0),
                                              ([17, 40, 99, 5000, 333], 5, 100), (list(range(0, 200, 7)) * 3, 0, 0)])
@pytest.mark.parametrize("shape", [(64, 1, 128), (48, 2, 128), (17, 1, 128), (136, 8, 128), (24, 2, 64), (64, 1, 64),
                                   (128, 8, 64), (9, 1, 256), (64, 1, 256), (48, 4, 256)])
def test_many_heads_in_splits_and_windows(cuda_device, shape, lens, sink, recent):
    """More heads per KV head than a warp's tile of eight: tiles, replicas and boxes of every kind."""
    Inputs(cuda_device, lens, *shape, seed=len(lens), sink=sink, recent=recent).check()


@pytest.mark.parametrize("batch", [19, 76, 151, 152, 153, 160, 161])
@pytest.mark.parametrize("shape", [(8, 2, 128), (9, 3, 64), (8, 8, 128), (12, 1, 256)])
def test_about_one_short_request_per_cta(cuda_device, batch, shape):
    """Around the batch sizes at which every piece of a request still gets a CTA of its own."""
    lens = [(0, 1, 64, 65, 128, 129, 16, 200, 0, 33, 7)[(b * b + b // 5) % 11] for b in range(batch)]
    Inputs(cuda_device, lens, *shape, seed=batch).check()
    Inputs(cuda_device, [100] * batch, *shape, seed=batch, sink=4, recent=70).check()


@pytest.mark.parametrize("Hq,H,D", [(1000, 1000, 64), (130, 65, 128)])
def test_many_kv_heads(cuda_device, Hq, H, D):
    """More (request, head group) items than CTAs from few requests, and about as many."""
    Inputs(cuda_device, [100, 0, 17], Hq, H, D, seed=H).check()
    Inputs(cuda_device, [33], Hq, H, D, seed=H).check()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("spread", [0, 12, 40])
@pytest.mark.parametrize("odd", [False, True])
def test_scales_of_pages(cuda_device, shape, spread, odd):
    """Pages whose scales differ by little, by 2^24 and by 2^80; powers of two or not."""
    Inputs(cuda_device, [70, 333, 17, 2500], *shape, scale=2.0 ** -spread / 8, seed=5, spread=spread, odd_scales=odd).check()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("k_exp,v_exp", [(-100, -100), (-100, 100), (60, -100), (60, 100)])
def test_least_and_large_scales(cuda_device, shape, k_exp, v_exp):
    """The least scales that a store writes, and large ones; the queries make ordinary logits of them."""
    x = Inputs(cuda_device, [70, 333, 17, 2500], *shape, seed=20, q_scale=2.0 ** (-7 - k_exp))
    for n, e in (("k", k_exp), ("v", v_exp)):
        x.s[n] = torch.exp2(torch.randint(e, e + 3, x.s[n].shape, generator=torch.Generator().manual_seed(e + 200)).float())
    x.upload()
    x.check()


# Shapes whose warps share a head's pages and shapes where each has its own, with one tile of heads and with many.
EVERY_SPLIT = SHAPES + [(64, 8, 128), (32, 8, 64), (64, 1, 128), (64, 1, 64), (64, 1, 256), (48, 4, 256)]


@pytest.mark.parametrize("shape", EVERY_SPLIT)
@pytest.mark.parametrize("lens,sink,recent", [([70, 0, 333, 17, 2500], 0, 0), ([20011], 0, 0), ([9000, 1, 4095], 0, 0),
                                              ([330] * 160, 0, 0), ([17, 40, 99, 5000, 333], 5, 100)])
def test_values_near_the_largest(cuda_device, shape, lens, sink, recent):
    """Values up to 448 2^119 = 0.875 2^128 of one sign, their weights nearly the same: the averages are finite, though the
    sums of two values are not. (Positive codes: only averages this large could overflow on the way.)"""
    x = Inputs(cuda_device, lens, *shape, seed=24, sink=sink, recent=recent, q_scale=0.01)
    x.codes["v"] &= 0x7F
    x.s["v"] = torch.exp2(torch.randint(118, 120, x.s["v"].shape, generator=torch.Generator().manual_seed(24)).float())
    x.upload()
    x.check()


@pytest.mark.parametrize("shape", EVERY_SPLIT)
@pytest.mark.parametrize("recent", [0, 1])
def test_large_queries_over_keys_of_the_least_scale(cuda_device, shape, recent):
    """Queries near 2^122 over K scales of 2^-100: the logits are some 2^30, the products with the codes alone beyond fp32.
    One kept token has all the weight, whatever its logit. Of more, whose logits and partial log-sum-exps are rounded in
    steps of 2^7, no weight is known, but that they are an average's: with A the largest |v_j| of a dim, the output lies
    within min_j v_j and max_j v_j but for (2^-11 + (n + 64) 2^-23) A (weights in fp16, sums) and the rounding to bf16."""
    lens = [1, 40, 0, 5000, 9000] if recent else [70, 0, 333, 17, 5000]
    x = Inputs(cuda_device, lens, *shape, seed=25, recent=recent, q_scale=2.0 ** 120)
    x.s["k"] = torch.full_like(x.s["k"], 2.0 ** -100)
    x.upload()
    out, lse = x.run()
    _, rlse, _, ltol = x.bounds()
    got = lse.double().cpu().numpy()
    empty = np.isneginf(rlse)
    assert (np.isneginf(got) == empty).all()
    assert (np.abs(np.where(empty, 0, got) - np.where(empty, 0, rlse)) <= ltol).all()
    v, got = x.value("v"), out.double().cpu().numpy()
    assert np.isfinite(got).all()
    for b, L in enumerate(lens):
        j = op.kept_positions(L, 0, recent)
        if len(j) == 0:
            assert (got[b] == 0).all()
            continue
        kept = np.repeat(v[x.table.numpy()[b, j // 16], :, j % 16], x.Hq // x.H, axis=1)
        lo, hi, far = kept.min(0), kept.max(0), np.abs(kept).max(0)
        tol = (2.0 ** -11 + (len(j) + 64) * 2.0 ** -23 + 2.0 ** -8 * (1 + 2.0 ** -7)) * far
        assert (got[b] >= lo - tol).all() and (got[b] <= hi + tol).all()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("scale,q_scale", [(0.0, 1.0), (-0.07, 1.0), (1.0, 0.1), (1e-3, 300.0), (1e20, 1e-21), (1e-9, 1e8)])
def test_scales_of_queries(cuda_device, shape, scale, q_scale):
    Inputs(cuda_device, [70, 333, 17], *shape, scale=scale, q_scale=q_scale, seed=6).check()


@pytest.mark.parametrize("shape", SHAPES)
def test_query_rows_of_many_magnitudes(cuda_device, shape):
    """Dims of a query row between 2^-30 and 1 of its largest, zeros among them, and a row of zeros."""
    x = Inputs(cuda_device, [70, 333, 17], *shape, seed=7)
    g = torch.Generator().manual_seed(7)
    x.q_all.copy_((x.q_all.float() * torch.exp2(torch.randint(-30, 1, x.q_all.shape, generator=g).float())).to(torch.bfloat16))
    x.q_all[:, :, ::7] = 0
    x.q_all[1, 0] = 0
    x.upload()
    x.check()


@pytest.mark.parametrize("q_pad", [3, 9])
@pytest.mark.parametrize("shape", SHAPES)
def test_queries_as_columns_of_a_wider_tensor(cuda_device, q_pad, shape):
    Inputs(cuda_device, [70, 333, 17], *shape, q_pad=q_pad, seed=5).check()


@pytest.mark.parametrize("shape", SHAPES)
def test_rising_logits_move_the_maximum(cuda_device, shape):
    """Every later page beats all before it, in its logits and in its V scale: maxima and references move at each."""
    Hq, H, D = shape
    x = Inputs(cuda_device, [1500], Hq, H, D, seed=7)
    x.q_all.copy_(x.q_all.abs())
    pages = x.table[0, :94].long()
    x.codes["k"][pages] &= 0x7F  # positive
    x.codes["k"][pages[-1], :, 12:] = 0x7F
    ramp = 2.0 ** -12 * (1 + torch.arange(94).float())
    x.s["k"][pages] = ramp[:, None].expand(-1, H).clone()
    x.s["v"][pages] = torch.exp2(torch.arange(94).float() / 4 - 20)[:, None].expand(-1, H).clone()
    x.upload()
    x.check()


@pytest.mark.parametrize("shape", SHAPES)
def test_stretches_without_a_finite_logit(cuda_device, shape):
    """Keys whose logits overflow to -inf, whole pages of them, carry no weight wherever the work is cut; a row of
    nothing else is empty."""
    Hq, H, D = shape
    lens = [40, 320, 5000, 33]
    x = Inputs(cuda_device, lens, Hq, H, D, seed=8, scale=4.0, q_scale=0.02)
    x.q_all[:, :, 0] = 1.0
    whole = {0: (0, 2), 1: (0, 20), 2: (40, 290), 3: (2, 3)}  # pages
    for b, (lo, hi) in whole.items():
        p = x.table[b, lo:hi].long()
        c = x.codes["k"][p]
        c[..., 0] = torch.where(c[..., 0] == 0x7F, c[..., 0], torch.full_like(c[..., 0], 0xFE))  # -448
        c[..., 1:] = torch.where(c[..., 1:] == 0x7F, c[..., 1:], torch.zeros_like(c[..., 1:]))
        x.codes["k"][p] = c
        x.s["k"][p] = 2.0 ** 119                                 # times 4: beyond fp32
    x.upload()
    out, lse = x.run()
    # What is left: the other pages in their order.
    y = Inputs(cuda_device, list(lens), Hq, H, D, seed=8, scale=4.0, q_scale=0.02)
    y.codes, y.s, y.q_all = x.codes, x.s, x.q_all
    y.q = y.q_all[:, :Hq]
    for b, (lo, hi) in whole.items():
        n = -(-lens[b] // 16)
        left = torch.cat([x.table[b, :lo], x.table[b, hi:n]])
        y.table[b, :len(left)] = left
        y.lens[b] = lens[b] - sum(min(16, lens[b] - 16 * p) for p in range(lo, hi))
    ref, rlse, tol, ltol = y.bounds()
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    empty = np.isneginf(rlse)
    got = lse.double().cpu().numpy()
    assert empty[1].all() and (np.isneginf(got) == empty).all() and bool((out[1] == 0).all())
    assert (np.abs(np.where(empty, 0, got) - np.where(empty, 0, rlse)) <= ltol).all()


@pytest.mark.parametrize("shape", SHAPES)
def test_nan_in_a_kept_value_stays_in_its_column(cuda_device, shape):
    Hq, H, D = shape
    x = Inputs(cuda_device, [50, 50], Hq, H, D, seed=9)
    want = torch.zeros(2, Hq, D, dtype=torch.bool)
    for dim in (7, 24, D - 1):
        x.codes["v"][x.table[0, 1].long(), H - 1, 4, dim] = 0x7F
        want[0, (H - 1) * (Hq // H):, dim] = True
    x.upload()
    out, lse = x.run()
    assert torch.equal(torch.isnan(out).cpu(), want) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_query_row_that_is_not_finite_is_nan(cuda_device, value):
    x = Inputs(cuda_device, [50, 0, 3000], 8, 2, 128, seed=10)
    x.q_all[:, 3, 17] = value
    x.upload()
    out, lse = x.run()
    bad = torch.zeros(3, 8, dtype=torch.bool)
    bad[0, 3] = bad[2, 3] = True
    assert torch.equal(torch.isnan(out).all(2).cpu(), bad) and torch.equal(torch.isnan(out).any(2).cpu(), bad)
    assert bool((out[1] == 0).all()) and bool(torch.isneginf(lse[1]).all())


@pytest.mark.parametrize("shape", SHAPES)
def test_no_lse(cuda_device, shape):
    x = Inputs(cuda_device, [70, 0, 333], *shape, seed=10)
    a, _ = x.run()
    b, _ = x.run(lse=False)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("shape", SHAPES)
def test_one_workspace_for_other_lengths_streams_and_caches(cuda_device, shape):
    """Calls in a row share a workspace, one over a bf16 cache among them; some run on another stream."""
    Hq, H, D = shape
    x = Inputs(cuda_device, [5000, 3], Hq, H, D, seed=11)
    y = Inputs(cuda_device, [7, 2500], Hq, H, D, seed=12)
    ws = torch.zeros(max(x.ws.numel(), se.se_paged_decode_workspace_size(2, Hq, H, D, D)), dtype=torch.uint8, device=cuda_device)
    want, _ = x.run()
    y.check()
    k = torch.randn(400, H, 16, D, device=cuda_device).to(torch.bfloat16)
    v = k.clone()
    kv = se.paged_kv(k, v, None)
    out = torch.empty(2, Hq, D, dtype=torch.bfloat16, device=cuda_device)
    table = torch.arange(400, dtype=torch.int32, device=cuda_device).view(2, 200)
    lens = torch.tensor([3000, 77], dtype=torch.int32, device=cuda_device)
    s = torch.cuda.Stream()
    for _ in range(3):
        se.se_paged_decode(kv, x.dq, table, lens, 0.1, out, None, ws)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            y.run(ws=ws)
        got, _ = x.run(ws=ws, stream=s)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("shape", SHAPES)
def test_bad_pages_and_lengths_are_reported_and_skipped(cuda_device, shape):
    x = Inputs(cuda_device, [64, 40, 33, 16], *shape, seed=13)
    y = Inputs(cuda_device, [48, 40, 33, 16], *shape, seed=13)
    y.codes, y.s, y.q_all, y.q = x.codes, x.s, x.q_all, x.q
    y.table = x.table.clone()
    y.table[0, 1:3] = x.table[0, 2:4]  # request 0 without its second page
    ref, rlse, tol, ltol = y.bounds()
    for bad in (-1, x.codes["k"].shape[0], 2**31 - 1):
        x.dt[0, 1] = bad
        out, lse = x.run()
        assert se.se_read_device_error(clear=True) == se.DEVERR_PAGE_RANGE
        assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
        assert (np.abs(lse.double().cpu().numpy() - rlse) <= ltol).all()
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


@pytest.mark.parametrize("shape", [(2, 1, 64), (2, 1, 256)])
def test_largest_batches(cuda_device, shape):
    g = np.random.default_rng(1)
    Inputs(cuda_device, g.integers(0, 24, 4096).tolist(), *shape, seed=16).check()


def test_a_cache_of_more_than_two_to_the_31_bytes(cuda_device):
    """Rows written to, read from and attended to in the pages at both ends of a 4.6 GB cache."""
    dev = cuda_device
    H, D, Hq, pages = 8, 128, 16, 140000
    k, v = (torch.empty(pages, H, 16, D, dtype=F8, device=dev) for _ in range(2))
    ks, vs = (torch.empty(pages, H, device=dev) for _ in range(2))
    assert k.numel() > 2 ** 31
    n = [300, 77]
    ids = [[pages - 1 - i for i in range(19)], [0, pages - 20, 1, pages // 2, pages - 21]]
    table = torch.zeros(2, 19, dtype=torch.int32)
    for b in range(2):
        table[b, :len(ids[b])] = torch.tensor(ids[b], dtype=torch.int32)
    slots = torch.tensor([ids[b][j // 16] * 16 + j % 16 for b in range(2) for j in range(n[b])], dtype=torch.int32)
    g = torch.Generator().manual_seed(17)
    kn, vn = (torch.randn(sum(n), H, D, generator=g).to(torch.bfloat16) for _ in range(2))
    kv = se.paged_kv8(k, v, ks, vs)
    se.se_paged_kv8_store(kv, kn.to(dev), vn.to(dev), slots.to(dev))
    back = [torch.empty(sum(n), H, D, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    start = torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device=dev)
    se.se_paged_kv8_load(kv, table.to(dev), start, *back)
    # Each element within half a step of e4m3 of its row (2^-4), or of its page's least steps.
    for x, y in zip((kn, vn), back):
        x, y = x.float(), y.float().cpu()
        assert bool(((x - y).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 * 2.0 ** -6).all())
    q = torch.randn(2, Hq, D, generator=g).to(torch.bfloat16)
    out = torch.empty(2, Hq, D, dtype=torch.bfloat16, device=dev)
    ws = torch.zeros(se.se_paged_kv8_decode_workspace_size(2, Hq, H, D), dtype=torch.uint8, device=dev)
    se.se_paged_kv8_decode(kv, q.to(dev), table.to(dev), torch.tensor(n, dtype=torch.int32, device=dev), 0.1, out, None, ws)
    for b in range(2):
        rows = slice(0, n[0]) if b == 0 else slice(n[0], sum(n))
        kk, vv = (t[rows].double().cpu().repeat_interleave(Hq // H, 1) for t in back)
        w = torch.softmax(0.1 * torch.einsum("ad,nad->an", q[b].double(), kk), 1)
        ref, mag = torch.einsum("an,nad->ad", w, vv), torch.einsum("an,nad->ad", w, vv.abs())
        assert bool(((out[b].double().cpu() - ref).abs() <= (2.0 ** -11 + 1e-4) * mag + 2.0 ** -8 * ref.abs() * 1.01).all())


@pytest.mark.parametrize("shape", SHAPES)
def test_calls_at_once_on_two_streams(cuda_device, shape):
    """Calls that share neither workspace nor outputs may overlap; their results stay."""
    x = Inputs(cuda_device, [5000, 3, 700], *shape, seed=21)
    y = Inputs(cuda_device, [7, 2500, 64], *shape, seed=22)
    want = [t.run()[0] for t in (x, y)]
    outs = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for t, o, st in zip((x, y), outs, streams):
            se.se_paged_kv8_decode(t.kv, t.dq, t.dt, t.dl, t.scale, o, None, t.ws, stream=st)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(w.view(torch.int16), o.view(torch.int16))


def test_a_view_keeps_its_tensors(cuda_device):
    x = Inputs(cuda_device, [5000, 3, 700], 8, 2, 128, seed=23)
    want, _ = x.run()
    x.kv = se.paged_kv8(x.d["k"].clone(), x.d["v"].clone(), x.ds["k"].clone(), x.ds["v"].clone())
    # What was freed would be handed out again here.
    taken = [torch.full_like(t.view(torch.uint8), 0x7F) for d in (x.d, x.ds) for t in d.values()]
    got, _ = x.run()
    assert len(taken) == 4 and torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_binding_checks(cuda_device):
    x = Inputs(cuda_device, [5, 6], 8, 2, 128, seed=15)
    out = torch.empty(2, 8, 128, dtype=torch.bfloat16, device=cuda_device)
    lse = torch.empty(2, 8, device=cuda_device)
    good = dict(kv=x.kv, q=x.dq, block_table=x.dt, seq_lens=x.dl, sm_scale=0.1, out=out, out_lse=lse, workspace=x.ws)
    se.se_paged_kv8_decode(**good)
    for name, bad, kind in [("q", x.dq[0], ValueError), ("q", x.dq.float(), TypeError), ("q", x.q, ValueError),
                            ("q", x.dq[:, :, :64], ValueError), ("block_table", x.dt[:1], ValueError),
                            ("seq_lens", x.dl[:1], ValueError), ("seq_lens", x.dl.long(), TypeError),
                            ("out", out[:1], ValueError), ("out", out.float(), TypeError), ("out_lse", lse[:1], ValueError),
                            ("out_lse", lse.half(), TypeError), ("workspace", x.ws[:8], se.SparseEngineError),
                            ("workspace", None, se.SparseEngineError), ("sm_scale", float("nan"), se.SparseEngineError)]:
        with pytest.raises(kind):
            se.se_paged_kv8_decode(**{**good, name: bad})
    with pytest.raises(se.SparseEngineError, match="sink_tokens without"):
        se.se_paged_kv8_decode(**good, sink_tokens=4)
