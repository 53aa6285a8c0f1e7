"""Dense paged decode where a long stretch of a request carries no finite logit: keys that make the logits
-inf, and pages that are skipped because their ids are out of range. What is left has to come out as if the
stretch were not there, wherever the work is cut.

A logit is -inf where a key holds -3.3e38 in its last dim against a query's 1 and sm_scale is 4: the scaled
product exceeds fp32 by a rounded multiplication, whatever the order of the sum. Heads with a 0 there see the
same tokens as ordinary ones. The next to last dim shifts a token's logits: up, so that the running maximum has
to move, or far down, where a base of 0 would leave no weight that fp32 can hold; the one before it shifts those
of the heads that a test chooses.

The bounds are those of the other decode tests, over the tokens whose logits are finite: with
dz = (D + 8) 2^-23 max_j sum_c |s q_c k_jc| and A = sum_j alpha_j |v_j|,
    |out - exact| <= (2^-8 + 2 dz + (n + 64) 2^-23) A + 2^-8 |exact| (1 + 2^-7) + 2^-133,
    |lse - exact| <= dz + (n + 64) 2^-23 + 2^-21 (1 + |exact|).
"""
import pytest
import torch

import sparse_decode_attention_quest_gb300 as se

pytestmark = pytest.mark.gpu

SCALE = 4.0
LOWEST = -3.3e38


@pytest.fixture(autouse=True)
def _no_device_errors(se_lib, cuda_device):
    se.se_read_device_error(clear=True)
    yield
    assert se.se_read_device_error(clear=True) == 0


class Requests:
    def __init__(self, dev, lens, Hq, H, D, seed):
        g = torch.Generator().manual_seed(seed)
        self.dev, self.lens, self.Hq, self.H, self.D = dev, lens, Hq, H, D
        self.latent = D == 576
        self.Dv = 512 if self.latent else D
        n = [-(-x // 16) for x in lens]
        self.table = torch.zeros(len(lens), max(n), dtype=torch.int32)
        perm = torch.randperm(sum(n), generator=g).int()
        for b, m in enumerate(n):
            self.table[b, :m] = perm[sum(n[:b]):sum(n[:b]) + m]
        shape = (sum(n), H, 16, D)
        self.k = (torch.randn(shape, generator=g) * 0.03).to(torch.bfloat16)
        self.k[..., D - 3:] = 0
        self.v = None if self.latent else torch.randn(shape, generator=g).to(torch.bfloat16)
        self.q = torch.randn(len(lens), Hq, D, generator=g).to(torch.bfloat16)
        self.q[..., D - 3] = 0
        self.q[..., D - 2:] = 1
        self.dropped = [torch.zeros(x, dtype=torch.bool) for x in lens]  # of skipped pages
        self.masked = [torch.zeros(x, dtype=torch.bool) for x in lens]   # by their keys

    def _set(self, b, lo, hi, dim, value):
        j = torch.arange(lo, hi)
        self.k[self.table[b, j // 16].long(), :, j % 16, dim] = value

    def mask(self, b, lo, hi):
        self._set(b, lo, hi, self.D - 1, LOWEST)
        self.masked[b][lo:hi] = True

    def shift(self, b, lo, hi, by, dim=-2):
        self._set(b, lo, hi, self.D + dim, by / SCALE)

    def rows(self, b):
        """Keys and values [H][tokens][..] of request b, in fp64 on the GPU."""
        j = torch.arange(self.lens[b])
        take = lambda t: t[self.table[b, j // 16].long(), :, j % 16].to(self.dev).double().transpose(0, 1)
        k = take(self.k)
        return k, k[..., :512] if self.latent else take(self.v)

    def run(self, table=None):
        dk = self.k.to(self.dev)
        dv = None if self.latent else self.v.to(self.dev)
        B = len(self.lens)
        out = torch.full((B, self.Hq, self.Dv), 77.0, dtype=torch.bfloat16, device=self.dev)
        lse = torch.full((B, self.Hq), 77.0, device=self.dev)
        ws = torch.zeros(se.se_paged_decode_workspace_size(B, self.Hq, self.H, self.D, self.Dv), dtype=torch.uint8,
                         device=self.dev)
        se.se_paged_decode(se.paged_kv(dk, dv, None, self.Dv), self.q.to(self.dev),
                           (self.table if table is None else table).to(self.dev),
                           torch.tensor(self.lens, dtype=torch.int32, device=self.dev), SCALE, out, lse, ws)
        torch.cuda.synchronize()
        return out.double(), lse.double()

    def check(self, out, lse):
        G = self.Hq // self.H
        for b in range(len(self.lens)):
            k, v = self.rows(b)
            q = self.q[b].to(self.dev).double().view(self.H, G, self.D)
            seen = ~self.dropped[b][None] & ~(self.masked[b][None] & (self.q[b, :, -1:] != 0))
            seen = seen.to(self.dev).view(self.H, G, -1)
            z = torch.where(seen, SCALE * q @ k.transpose(1, 2), -torch.inf)
            rlse = torch.logsumexp(z, -1)
            w = torch.where(seen, torch.exp(z - torch.where(torch.isinf(rlse), 0.0, rlse)[..., None]), 0.0)
            ref, mag = w @ v, w @ v.abs()
            zmag = torch.where(seen, SCALE * q.abs() @ k.abs().transpose(1, 2), 0.0).amax(-1)
            n = seen.sum(-1)
            dz = (self.D + 8) * 2.0 ** -23 * zmag
            got, glse = out[b].view(ref.shape), lse[b].view(rlse.shape)
            tol = (2.0 ** -8 + 2 * dz + (n + 64) * 2.0 ** -23)[..., None] * mag + 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -7)
            bad = ~((got - ref).abs() <= tol + 2.0 ** -133)
            assert not bool(bad.any()), f"request {b}: {int(bad.any(-1).sum())} heads, off by {(got - ref).abs().max():.3g}"
            none = n == 0
            assert torch.equal(torch.isneginf(glse), none), f"request {b}: lse {glse.flatten()[:4].tolist()}"
            ltol = dz + (n + 64) * 2.0 ** -23 + 2.0 ** -21 * (1 + torch.where(none, 0.0, rlse).abs())
            assert bool(((torch.where(none, 0.0, glse - rlse)).abs() <= ltol).all()), f"request {b}"


SHAPES = [(16, 1, 576), (64, 1, 576), (8, 2, 128), (16, 1, 64)]
# 160 requests: one or two to a CTA, most of them whole. Two long ones: cut into some 150 segments.
BATCHES = {"whole": [300] * 160, "split": [20011, 9000]}


def _mask(x, kind):
    for b, n in enumerate(x.lens):
        if kind == "split":
            for lo, hi in [(0, 64 + 66 * b), (200, 3000), (3100, 3300), (6000, 6064), (n - 900, n)]:
                x.mask(b, lo, hi)
        else:
            x.mask(b, 0, (0, 63, 64, 65, 130, 192, n)[b % 7])


@pytest.mark.parametrize("heads", ["all", "half"])
@pytest.mark.parametrize("kind", list(BATCHES))
@pytest.mark.parametrize("shape", SHAPES)
def test_masked_stretches(cuda_device, shape, kind, heads):
    x = Requests(cuda_device, BATCHES[kind], *shape, seed=1)
    _mask(x, kind)
    if heads == "half":
        x.q[:, ::2, -1] = 0
    x.check(*x.run())


@pytest.mark.parametrize("base,peaks", [(0.0, 40.0), (-20.0, None), (-20.0, 40.0), (-400.0, None), (-400.0, -380.0)])
@pytest.mark.parametrize("kind", list(BATCHES))
@pytest.mark.parametrize("shape", SHAPES)
def test_what_follows_a_masked_stretch_is_far_off(cuda_device, shape, kind, base, peaks):
    """Logits well below 0, some beyond what a weight against a base of 0 could hold, and later tokens that
    move the running maxima."""
    x = Requests(cuda_device, BATCHES[kind], *shape, seed=2)
    _mask(x, kind)
    x.q[:, ::3, -1] = 0
    for b, n in enumerate(x.lens):
        x.shift(b, 0, n, base)
        if peaks is not None:
            for lo in range(250, n, 2000):
                x.shift(b, lo, lo + 3, peaks)
    x.check(*x.run())


@pytest.mark.parametrize("kind", list(BATCHES))
@pytest.mark.parametrize("shape", SHAPES)
def test_other_heads_move_their_maxima(cuda_device, shape, kind):
    """Behind a masked stretch every head sums logits near -20; then a quarter of the heads meets some near 20, which
    takes nothing from the sums of the others."""
    x = Requests(cuda_device, BATCHES[kind], *shape, seed=4)
    _mask(x, kind)
    x.q[:, 1::4, -3] = 1
    for b, n in enumerate(x.lens):
        x.shift(b, 0, n, -20.0)
        for lo in range(270, n, 500):
            x.shift(b, lo, lo + 2, 40.0, dim=-3)
    x.check(*x.run())


@pytest.mark.parametrize("kind", list(BATCHES))
@pytest.mark.parametrize("shape", SHAPES)
def test_skipped_pages(cuda_device, shape, kind):
    """Pages with ids out of range at a request's start and, in long ones, over whole stretches."""
    x = Requests(cuda_device, BATCHES[kind], *shape, seed=3)
    table = x.table.clone()
    for b, n in enumerate(x.lens):
        pages = -(-n // 16)
        for lo, hi in [(0, 4 + b % 9), (30, 190), (200, 204)]:
            table[b, lo:min(hi, pages)] = (-1, x.k.shape[0], 2 ** 31 - 1)[b % 3]
            x.dropped[b][lo * 16:hi * 16] = True
        x.shift(b, 0, n, -100.0 * (b % 2))
    got = x.run(table)
    assert se.se_read_device_error(clear=True) == se.DEVERR_PAGE_RANGE
    x.check(*got)
