"""The 8-bit cache as a serving loop uses it: prompts admitted, turned by their positions, stored and read back; decode
steps (live and recorded) that take pages, turn and write rows and attend; requests that leave and come.

Codes and scales are compared exactly with the run-by-run simulation over the turned rows that the GPU stored, rows read
back exactly with the codes' values, and outputs with the bounds of the decode tests over those values (half a step of
fp16 a weight, one rounding of the output)."""
import numpy as np
import pytest
import torch

import oracle.kv8 as k8
import oracle.paged as op
import sparse_decode_attention_quest_gb300 as se
from sparse_decode_attention_quest_gb300.pipeline import DenseAttention, PagedCache, Rotary

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_errors(se_lib, cuda_device):
    se.se_read_device_error(clear=True)
    yield
    assert se.se_read_device_error(clear=True) == 0


def _bf16(shape, g, dev):
    return torch.randn(shape, generator=g).to(torch.bfloat16).to(dev)


def _codes(t):
    return t.view(torch.uint8).cpu().numpy().copy()


class Model:
    """The cache's contents by the simulation, from what the GPU was given to store."""

    def __init__(self, cache):
        self.c = cache
        self.codes = {"k": _codes(cache.k), "v": _codes(cache.v)}
        self.scale = {"k": cache.k_scale.cpu().numpy().copy(), "v": cache.v_scale.cpu().numpy().copy()}

    def store(self, k, v):
        slots = self.c.slot_map[:k.shape[0]].tolist()
        for n, x in (("k", k), ("v", v)):
            k8.store(self.codes[n], self.scale[n], x.double().cpu().numpy(), slots)

    def check(self):
        for n, t, s in (("k", self.c.k, self.c.k_scale), ("v", self.c.v, self.c.v_scale)):
            np.testing.assert_array_equal(s.cpu().numpy(), self.scale[n])
            np.testing.assert_array_equal(_codes(t), self.codes[n])

    def value(self, n):
        return k8.values(self.codes[n], self.scale[n])

    def check_attention(self, q, lens, sink=0, recent=0):
        out, lse = self.c.attention.out, self.c.attention.lse
        D = q.shape[-1]
        ref, rlse, mag, zmag = op.decode(self.value("k"), self.value("v"), self.c.block_table.cpu().numpy(), lens,
                                         q.double().cpu().numpy(), self.c.attention.sm_scale, D, sink, recent)
        # Rows of unit variance: M sum_c |k_jc| is below 2^9 max_j sum_c |q_c k_jc|, 2^-32 of it below a rounding of fp32.
        dz = (D + 13) * 2.0 ** -23 * zmag
        n = np.array(lens)[:, None]
        tol = (2.0 ** -11 + 2 * dz + (n + 64) * 2.0 ** -23)[..., None] * mag + 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7)
        tol = tol + (n * 2.0 ** -39 * 448)[..., None] * max(float(x.max()) for x in (self.scale["v"],))
        assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
        ltol = dz + (n + 64) * 2.0 ** -23 + 2.0 ** -21 * (1 + np.abs(np.where(np.isinf(rlse), 0, rlse)))
        got = lse.double().cpu().numpy()
        assert (np.isneginf(got) == np.isneginf(rlse)).all()
        fine = ~np.isneginf(rlse)
        assert (np.abs(got - np.where(fine, rlse, 0))[fine] <= ltol[fine]).all()


SHAPES = {"gqa": dict(num_q_heads=8, num_kv_heads=2, head_dim=128), "narrow": dict(num_q_heads=10, num_kv_heads=5, head_dim=64),
          "wide": dict(num_q_heads=6, num_kv_heads=3, head_dim=256)}


def _qkv(T, kw, g, dev):
    """Query, key and value rows as columns of a fused projection's output."""
    hq, h, d = kw["num_q_heads"], kw["num_kv_heads"], kw["head_dim"]
    fused = _bf16((T, hq + 2 * h, d), g, dev)
    return fused, fused[:, :hq], fused[:, hq:hq + h], fused[:, hq + h:]


@pytest.mark.parametrize("shape", list(SHAPES))
def test_prompts_steps_and_rows_back(cuda_device, shape):
    dev, kw = cuda_device, SHAPES[shape]
    H, D = kw["num_kv_heads"], kw["head_dim"]
    g = torch.Generator().manual_seed(1)
    cache = PagedCache(90, 5, 400, max_new_tokens=600, device=dev, eight_bit=True, **kw)
    rotary = Rotary(D // 2, dev, offset=D // 4, scaling="yarn", factor=4.0, original_len=100)
    model = Model(cache)
    lens = [130, 0, 47, 300, 16]
    cache.extend(torch.tensor(lens, dtype=torch.int32, device=dev))
    fused, q, k, v = _qkv(sum(lens) + 3, kw, g, dev)
    before = fused.clone()
    cache.rotate(rotary, q, k)
    w, amp = k8.frequencies(D // 2, 10000.0, "yarn", 4.0, 100)
    pos = np.concatenate([np.arange(n) for n in lens])
    T = sum(lens)
    x = before[:T, :kw["num_q_heads"] + H].double().cpu().numpy()
    want = k8.rotary(x, pos, w, D // 4, False, False, amp)
    lo, hi = D // 4, D // 4 + D // 2
    part = np.abs(x[..., lo:hi])
    tol = (2.0 ** -22 + 6 * 2.0 ** -23) * amp * (part + np.roll(part, D // 4, -1)) + 2.0 ** -8 * np.abs(want[..., lo:hi]) * 1.01
    got = fused[:T, :kw["num_q_heads"] + H].double().cpu().numpy()
    assert (np.abs(got - want)[..., lo:hi] <= tol).all()
    assert torch.equal(fused[T:], before[T:]) and torch.equal(v, before[:, kw["num_q_heads"] + H:])  # padding and values
    cache.store(k[:T], v[:T])
    model.store(k[:T], v[:T])
    model.check()
    # Whole requests back, and the last tokens of each.
    for firsts in (None, [100, 0, 40, 299, 0]):
        counts = [n - (0 if firsts is None else firsts[b]) for b, n in enumerate(lens)]
        start = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=dev)
        ko, vo = (torch.full((sum(counts) + 4, H, D), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(2))
        cache.load(start, ko, vo, None if firsts is None else torch.tensor(firsts, dtype=torch.int32, device=dev))
        for n, o in (("k", ko), ("v", vo)):
            ref, _ = k8.load(model.codes[n], model.scale[n], cache.block_table.cpu().numpy(), start.tolist(),
                             np.full(o.shape, 7.0), firsts)
            np.testing.assert_array_equal(o.double().cpu().numpy(), ref)
    # A few decode steps, over everything and over windows.
    for t in range(4):
        cache.extend(torch.ones(5, dtype=torch.int32, device=dev))
        lens = [n + 1 for n in lens]
        _, q, k, v = _qkv(5, kw, g, dev)
        cache.rotate(rotary, q, k)
        cache.store(k, v)
        model.store(k, v)
        window = (0, 0) if t % 2 else (5, 40)
        cache.attend(q, *window)
        model.check()
        model.check_attention(q, lens, *window)


@pytest.mark.parametrize("shape", list(SHAPES))
def test_recorded_steps_grow_the_cache(cuda_device, shape):
    """One recording of extend + rotate + store + attend, replayed over 20 steps: requests cross page borders, one gets
    no token in some steps, and the padded end of the batch of new tokens is left and skipped."""
    dev, kw = cuda_device, SHAPES[shape]
    hq, H, D = kw["num_q_heads"], kw["num_kv_heads"], kw["head_dim"]
    B, g = 5, torch.Generator().manual_seed(2)
    cache = PagedCache(80, B, 400, max_new_tokens=600, device=dev, eight_bit=True, **kw)
    rotary = Rotary(D, dev, interleaved=True)
    lens = [130, 0, 47, 300, 16]
    cache.extend(torch.tensor(lens, dtype=torch.int32, device=dev))
    _, _, k, v = _qkv(sum(lens), kw, g, dev)
    cache.store(k, v)
    model = Model(cache)
    new = torch.ones(B, dtype=torch.int32, device=dev)
    fused, q, k, v = _qkv(B + 2, kw, g, dev)   # two rows of padding
    qt, kt = torch.zeros(B + 2, hq, D, dtype=torch.bfloat16, device=dev), torch.zeros(B + 2, H, D, dtype=torch.bfloat16, device=dev)
    attended = torch.zeros(B, hq, D, dtype=torch.bfloat16, device=dev)
    stream = torch.cuda.Stream(device=dev)
    torch.cuda.synchronize()
    se.se_capture_begin(stream)
    cache.extend(new, stream)
    cache.rotate(rotary, q, k, qt, kt, stream)
    cache.store(kt, v, stream)
    cache.attend(attended, stream=stream)
    step = se.se_capture_end(stream)
    assert cache.lens.tolist() == lens  # nothing ran yet
    for t in range(20):
        counts = [1, 1, int(t % 3 == 0), 1, 2]
        new.copy_(torch.tensor(counts, dtype=torch.int32))
        fused.copy_(_bf16(fused.shape, g, dev))
        attended.copy_(_bf16(attended.shape, g, dev))
        qt.fill_(7.0)
        kt.fill_(7.0)
        torch.cuda.synchronize()
        step.launch(stream)
        stream.synchronize()
        n = sum(counts)
        assert bool((qt[n:] == 7.0).all()) and bool((kt[n:] == 7.0).all())
        want_q, want_k = torch.empty_like(qt), torch.empty_like(kt)
        rotary.apply(q, k, cache.positions[:B + 2], want_q, want_k)
        assert torch.equal(qt[:n], want_q[:n]) and torch.equal(kt[:n], want_k[:n])
        lens = [a + b for a, b in zip(lens, counts)]
        assert cache.lens.tolist() == lens
        model.store(kt, v)
        model.check()
        model.check_attention(attended, lens)


def test_pages_that_return_and_are_taken_again(cuda_device):
    """Requests leave, their pages go to others: a page's old scale does not outlive it, one that is cut keeps its own."""
    dev, kw = cuda_device, SHAPES["gqa"]
    g = torch.Generator().manual_seed(3)
    cache = PagedCache(13, 2, 200, max_new_tokens=200, device=dev, eight_bit=True, **kw)
    cache.extend(torch.tensor([100, 90], dtype=torch.int32, device=dev))
    _, _, k, v = _qkv(190, kw, g, dev)
    cache.store(k * 64, v * 64)
    model = Model(cache)
    cache.release(torch.tensor([21, 0], dtype=torch.int32, device=dev))
    lens = [21, 0]
    for counts in ([3, 70], [20, 5]):
        cache.extend(torch.tensor(counts, dtype=torch.int32, device=dev))
        _, q, k, v = _qkv(sum(counts), kw, g, dev)
        cache.store(k, v)
        model.store(k, v)
        lens = [a + b for a, b in zip(lens, counts)]
        cache.attend(q[:2])
        model.check()
        model.check_attention(q[:2], lens)
    cut, fresh = cache.block_table[0, 1], cache.block_table[1, 0]
    assert float(cache.k_scale[cut].min()) >= 0.25 and float(cache.k_scale[fresh].max()) <= 2.0 ** -5


def test_a_latent_cache_turns_its_last_dims(cuda_device):
    """Rotary positions before the bf16 latent cache: 64 of 576 dims, in place, then the store and the attention."""
    dev = cuda_device
    g = torch.Generator().manual_seed(4)
    cache = PagedCache(20, 2, 160, 16, 1, 576, 300, dev, latent=True, head_dim_v=512)
    rotary = Rotary(64, dev, offset=512, interleaved=True)
    lens = [60, 33]
    cache.extend(torch.tensor(lens, dtype=torch.int32, device=dev))
    k = _bf16((93, 1, 576), g, dev)
    before = k.clone()
    cache.rotate(rotary, None, k)
    assert torch.equal(k[..., :512], before[..., :512]) and not torch.equal(k[..., 512:], before[..., 512:])
    cache.store(k)
    q = _bf16((2, 16, 576), g, dev)
    rotary.apply(q, None, cache.lens - 1)
    out = cache.attend(q)
    ref, _, mag, _ = op.decode(cache.k.float().cpu().numpy(), None, cache.block_table.cpu().numpy(), lens,
                               q.float().cpu().numpy(), cache.attention.sm_scale, 512)
    assert (np.abs(out.double().cpu().numpy() - ref) <= (2.0 ** -8 + 1e-4) * mag + 2.0 ** -8 * np.abs(ref) * 1.01).all()


def test_eight_bits_stay_close_to_sixteen(cuda_device):
    """The same rows in both caches: keys and values are off by half a step of e4m3 (2^-4 of each, or 2^-10 of the page's
    scale), so that logits differ by at most dz = s sum_c |q_c| (2^-4 |k_c| + 2^-10 s_k) and outputs by
    2 dz (1 + dz) max |v| + 2^-4 |v| + 2^-10 s_v, beside the roundings of both."""
    dev = cuda_device
    g = torch.Generator().manual_seed(5)
    kw = dict(num_q_heads=8, num_kv_heads=2, head_dim=128)
    lens = torch.tensor([70, 33], dtype=torch.int32, device=dev)
    caches = [PagedCache(10, 2, 160, max_new_tokens=200, device=dev, eight_bit=e, **kw) for e in (False, True)]
    _, _, k, v = _qkv(103, kw, g, dev)
    k = k * 0.1
    q = _bf16((2, 8, 128), g, dev)
    for c in caches:
        c.extend(lens)
        c.store(k, v)
        c.attend(q)
    a, b = (c.attention.out.float() for c in caches)
    sk, sv = float(caches[1].k_scale[:8].max()), float(caches[1].v_scale[:8].max())
    dz = float(caches[0].attention.sm_scale * (q.float().abs().sum(2).max() * (2.0 ** -4 * k.float().abs().max() + 2.0 ** -10 * sk)))
    big = float(v.float().abs().max())
    assert float((a - b).abs().max()) <= 2 * dz * (1 + dz) * big + 2.0 ** -4 * big + 2.0 ** -10 * sv + 2.0 ** -7 * big


@pytest.mark.parametrize("shape", list(SHAPES))
def test_eight_bits_against_the_rows_themselves(cuda_device, shape):
    """Against 64 bits over the bf16 rows that were stored, bounded for each request and head. A value is off by half a
    step of e4m3: e(x) = max(2^-4 |x|, 2^-10 of its page's scale). Logits are then off by at most
    dz = s max_j sum_c |q_c| e(k_jc), weights by a factor within exp(+-2 dz), and the output by
    (exp(2 dz) - 1) sum_j w_j (|v_j| + e(v_j)) + sum_j w_j e(v_j), beside the kernel's own roundings (weights in fp16, sums, bf16).
    Outputs of zeros, of the other request or of the other sign are farther off than that."""
    dev, kw = cuda_device, SHAPES[shape]
    hq, H, D = kw["num_q_heads"], kw["num_kv_heads"], kw["head_dim"]
    g = torch.Generator().manual_seed(5)
    lens = [70, 33]
    cache = PagedCache(10, 2, 160, max_new_tokens=200, device=dev, eight_bit=True, **kw)
    k, v = (_bf16((103, H, D), g, dev) for _ in range(2))
    k = k * 0.1
    q = _bf16((2, hq, D), g, dev)
    cache.extend(torch.tensor(lens, dtype=torch.int32, device=dev))
    cache.store(k, v)
    out = cache.attend(q).double().cpu().numpy()
    table, s = cache.block_table.cpu().numpy(), cache.attention.sm_scale
    ref, tol = np.zeros_like(out), np.zeros_like(out)
    for b, n in enumerate(lens):
        page = table[b, np.arange(n) // 16]
        rows = slice(0, 70) if b == 0 else slice(70, 103)
        # [heads][tokens][dims], a KV head's for each of its query heads
        kk, vv = (np.repeat(x[rows].double().cpu().numpy().transpose(1, 0, 2), hq // H, 0) for x in (k, v))
        ks, vs = (np.repeat(x.double().cpu().numpy()[page].T, hq // H, 0)[:, :, None] for x in (cache.k_scale, cache.v_scale))
        qq = q[b].double().cpu().numpy()
        ek, ev = np.maximum(2.0 ** -4 * np.abs(kk), 2.0 ** -10 * ks), np.maximum(2.0 ** -4 * np.abs(vv), 2.0 ** -10 * vs)
        z = s * np.einsum("hd,hnd->hn", qq, kk)
        w = np.exp(z - z.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        dz = s * np.einsum("hd,hnd->hn", np.abs(qq), ek).max(1)[:, None]
        mag, off = (np.einsum("hn,hnd->hd", w, x) for x in (np.abs(vv), ev))
        ref[b] = np.einsum("hn,hnd->hd", w, vv)
        tol[b] = np.expm1(2 * dz) * (mag + off) + off + (2.0 ** -11 + (D + n + 64) * 2.0 ** -22) * (mag + off) * np.exp(2 * dz)
        tol[b] += 2.0 ** -8 * 1.01 * (np.abs(ref[b]) + tol[b])
    assert (np.abs(out - ref) <= tol).all()
    for wrong in (np.zeros_like(out), out[::-1], -out):
        for b in range(2):
            assert (np.abs(wrong[b] - ref[b]) > tol[b]).any()


def test_rows_of_neither_kind(cuda_device):
    cache = PagedCache(4, 1, 32, 8, 2, 128, 8, cuda_device, eight_bit=True)
    with pytest.raises(ValueError, match="neither is given"):
        cache.rotate(Rotary(128, cuda_device), None, None)


def test_refusals(cuda_device):
    dev = cuda_device
    for bad in (dict(latent=True, head_dim_v=512, head_dim=576, num_q_heads=16, num_kv_heads=1),
                dict(summary=True, head_dim=128, num_q_heads=8, num_kv_heads=2)):
        with pytest.raises(ValueError, match="8-bit"):
            PagedCache(4, 1, 32, max_new_tokens=8, device=dev, eight_bit=True, **bad)
    c = PagedCache(4, 1, 32, 8, 2, 128, 8, dev)
    rows = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device=dev)
    with pytest.raises(ValueError, match="not in 8 bits"):
        c.load(torch.zeros(2, dtype=torch.int32, device=dev), rows, rows)
    assert DenseAttention(c.kv, 1, 8, dev).eight_bit is False
