"""se_rotary on the GPU against fp64.

The angle is exact modulo a turn but for its rounding to 32 bits and to fp32 (2^-24 of half a turn: 2^-22 radians),
cosine and sine are good to 2 steps of 2^-24, amplitude, products and their difference add 4 of 2^-23 of the operands'
magnitudes, and the result is rounded to bf16 once. The frequencies, the library's and the oracle's, are off by
some steps of 2^-53, that is by 2^-49 of an angle:
    |y - exact| <= (2^-22 + 6 2^-23 + 2^-49 angle) amplitude (|x0| + |x1|) + 2^-8 |exact| (1 + 2^-7).
"""
import numpy as np
import pytest
import torch

import oracle.kv8 as k8
import sparse_decode_attention_quest_gb300 as se

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_errors(se_lib, cuda_device):
    se.se_read_device_error(clear=True)
    yield
    assert se.se_read_device_error(clear=True) == 0


def _rows(g, T, before, heads, behind, D):
    return torch.randn(T, before + heads + behind, D, generator=g).to(torch.bfloat16)


def _check(dev, positions, hq, hk, D, rot, offset=0, interleaved=False, inverse=False, in_place=False, fused=0,
           scaling=("none", 1.0, 0), valid=None, seed=0, stream=None):
    g = torch.Generator().manual_seed(seed)
    T = len(positions)
    freqs, amp = se.se_rotary_frequencies(rot, 10000.0, *scaling)
    w, amplitude = k8.frequencies(rot, 10000.0, *scaling)
    pos = torch.tensor(positions, dtype=torch.int32)
    n = torch.tensor([valid], dtype=torch.int32, device=dev) if valid is not None else None
    live = (np.arange(T) < (T if valid is None else valid)) & (np.array(positions) >= 0)
    args = {}
    sides = {}
    for name, heads in (("q", hq), ("k", hk)):
        if heads == 0:
            args[name] = args[name + "_out"] = None
            continue
        whole = _rows(g, T, fused, heads, fused, D)
        on = whole.to(dev)
        x = on[:, fused:fused + heads]
        out = None if in_place else torch.full((T, heads, D), 7.0, dtype=torch.bfloat16, device=dev)
        args[name], args[name + "_out"] = x, out
        sides[name] = (whole, on, x, out, heads)
    se.se_rotary(args["q"], args["k"], pos.to(dev), freqs.to(dev), args["q_out"], args["k_out"], rotary_offset=offset,
                 interleaved=interleaved, inverse=inverse, amplitude=amp, num_valid=n, stream=stream)
    torch.cuda.synchronize()
    for whole, on, x, out, heads in sides.values():
        src = whole[:, fused:fused + heads].double().numpy()
        got = (x if out is None else out).double().cpu().numpy()
        ref = k8.rotary(src, positions, w, offset, interleaved, inverse, amplitude)
        lo, hi = offset, offset + rot
        part = np.abs(src[..., lo:hi])
        mate = part.reshape(T, heads, -1, 2)[..., ::-1].reshape(part.shape) if interleaved else np.roll(part, rot // 2, -1)
        far = 2.0 ** -49 * np.abs(np.array(positions, dtype=np.float64))[:, None, None]  # the first frequency is the largest: 1
        tol = (2.0 ** -22 + 6 * 2.0 ** -23 + far) * amplitude * (part + mate) + 2.0 ** -8 * np.abs(ref[..., lo:hi]) * (1 + 2.0 ** -7)
        err = np.abs(got - ref)[..., lo:hi]
        assert (err[live] <= tol[live]).all(), f"off by {err[live].max():.3g}"
        # The other dims are copies; rows that are not live are as they were.
        np.testing.assert_array_equal(got[live][..., :lo], src[live][..., :lo])
        np.testing.assert_array_equal(got[live][..., hi:], src[live][..., hi:])
        np.testing.assert_array_equal(got[~live], src[~live] if out is None else np.full_like(src[~live], 7.0))
        # Nothing outside the rows of these heads changed.
        others = np.ones(on.shape[1], dtype=bool)
        others[fused:fused + heads] = False
        np.testing.assert_array_equal(on.double().cpu().numpy()[:, others], whole.double().numpy()[:, others])
        if out is not None:
            np.testing.assert_array_equal(x.double().cpu().numpy(), src)


LAYOUTS = [(4, 1, 128, 128, 0), (32, 8, 128, 64, 0), (3, 3, 64, 64, 0), (5, 2, 64, 32, 32), (2, 1, 256, 256, 0),
           (7, 1, 128, 96, 16), (10, 10, 128, 72, 0), (1, 1, 8, 8, 0), (1, 0, 16, 8, 8), (0, 2, 24, 8, 8), (16, 1, 576, 64, 512),
           (2, 2, 576, 576, 0), (300, 40, 64, 64, 0), (3, 5, 40, 40, 0)]


@pytest.mark.parametrize("hq,hk,D,rot,offset", LAYOUTS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_layouts(cuda_device, hq, hk, D, rot, offset, interleaved, in_place):
    _check(cuda_device, [0, 1, 5, 4096, 131071, 7, 1000000], hq, hk, D, rot, offset, interleaved, in_place=in_place, seed=hq)


@pytest.mark.parametrize("T", [1, 2, 3, 31, 152, 153, 2431, 2432, 2433, 5000])
def test_numbers_of_tokens(cuda_device, T):
    """One token a CTA up to 16 for every SM, several beyond."""
    g = np.random.default_rng(T)
    _check(cuda_device, g.integers(0, 200000, T).tolist(), 4, 2, 128, 128, seed=T)
    _check(cuda_device, g.integers(0, 200000, T).tolist(), 1, 1, 64, 16, 8, True, in_place=True, seed=T)


@pytest.mark.parametrize("fused", [1, 3])
@pytest.mark.parametrize("in_place", [False, True])
def test_columns_of_a_wider_tensor(cuda_device, fused, in_place):
    _check(cuda_device, list(range(100, 140)), 8, 2, 128, 128, fused=fused, in_place=in_place, seed=fused)
    _check(cuda_device, list(range(100, 140)), 3, 1, 64, 24, 16, fused=fused, in_place=in_place, inverse=True)


@pytest.mark.parametrize("scaling", [("linear", 4.0, 0), ("ntk", 8.0, 0), ("yarn", 4.0, 4096), ("yarn", 32.0, 8192)])
@pytest.mark.parametrize("inverse", [False, True])
def test_scaled_frequencies(cuda_device, scaling, inverse):
    _check(cuda_device, [0, 3, 500, 70000, 999999, 2**31 - 1], 4, 2, 128, 128, scaling=scaling, inverse=inverse)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("valid", [0, 1, 37, 38, 50, 100])
def test_rows_behind_the_last_valid_one_are_left(cuda_device, valid, in_place):
    _check(cuda_device, list(range(50)), 4, 1, 128, 64, valid=valid, in_place=in_place)


def test_rows_with_negative_positions_are_left(cuda_device):
    p = [3, -1, 8, -2**31, 0, -7] * 3
    _check(cuda_device, p, 4, 2, 64, 64)
    _check(cuda_device, p * 1000, 4, 2, 64, 64, in_place=True)


def test_turning_back(cuda_device):
    dev = cuda_device
    g = torch.Generator().manual_seed(4)
    x = torch.randn(64, 4, 128, generator=g).to(torch.bfloat16).to(dev)
    freqs = se.se_rotary_frequencies(128)[0].to(dev)
    pos = torch.arange(64, dtype=torch.int32, device=dev) * 999
    y, z = torch.empty_like(x), torch.empty_like(x)
    se.se_rotary(x, None, pos, freqs, y)
    se.se_rotary(y, None, pos, freqs, z, inverse=True)
    # Two roundings of 2^-8, and a pair's other value shares in the first one's.
    a, b = x.float().chunk(2, 2)
    size = torch.cat([torch.hypot(a, b)] * 2, 2)
    assert bool(((z - x).float().abs() <= 2.0 ** -7 * 1.01 * size).all())


@pytest.mark.parametrize("interleaved", [False, True])
def test_outputs_as_columns_of_a_wider_tensor(cuda_device, interleaved):
    dev = cuda_device
    g = torch.Generator().manual_seed(6)
    q, k = (torch.randn(37, h, 128, generator=g).to(torch.bfloat16).to(dev) for h in (6, 2))
    pos = (torch.arange(37, dtype=torch.int32) * 77).to(dev)
    freqs = se.se_rotary_frequencies(64)[0].to(dev)
    want = [torch.empty_like(t) for t in (q, k)]
    se.se_rotary(q, k, pos, freqs, *want, rotary_offset=32, interleaved=interleaved)
    wide = torch.full((37, 13, 128), 7.0, dtype=torch.bfloat16, device=dev)
    se.se_rotary(q, k, pos, freqs, wide[:, 1:7], wide[:, 9:11], rotary_offset=32, interleaved=interleaved)
    assert torch.equal(wide[:, 1:7], want[0]) and torch.equal(wide[:, 9:11], want[1])
    assert bool((wide[:, [0, 7, 8, 11, 12]] == 7.0).all())
    # One in place, the other not: the same bits, and dims that are not turned stay.
    mixed = q.clone()
    se.se_rotary(mixed, k, pos, freqs, None, wide[:, 9:11], rotary_offset=32, interleaved=interleaved)
    assert torch.equal(mixed, want[0]) and torch.equal(wide[:, 9:11], want[1])


def test_another_stream_and_a_recorded_step(cuda_device):
    dev = cuda_device
    s = torch.cuda.Stream(device=dev)
    _check(dev, [9, 8, 7], 4, 1, 128, 128, stream=s)
    freqs = se.se_rotary_frequencies(64)[0].to(dev)
    x, out = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=dev), torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=dev)
    pos = torch.zeros(3, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    se.se_capture_begin(s)
    se.se_rotary(None, x, pos, freqs, None, out, stream=s)
    step = se.se_capture_end(s)
    for i in range(3):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16))
        pos.copy_(torch.tensor([i, 100 * i, 12345], dtype=torch.int32))
        torch.cuda.synchronize()
        step.launch(s)
        s.synchronize()
        want = torch.empty_like(out)
        se.se_rotary(None, x, pos, freqs, None, want)
        assert torch.equal(out, want)


def test_rows_beyond_two_to_the_31_elements(cuda_device):
    """Tokens whose rows lie 2^31 elements and more from the first."""
    dev = cuda_device
    T, width = 60000, 40000
    x = torch.zeros(T, width, dtype=torch.bfloat16, device=dev)
    rows = x[:, :128].unflatten(1, (1, 128))
    g = torch.Generator().manual_seed(5)
    head = torch.randn(T, 1, 128, generator=g).to(torch.bfloat16).to(dev)
    rows.copy_(head)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    freqs = se.se_rotary_frequencies(128)[0].to(dev)
    se.se_rotary(rows, None, pos, freqs)
    want = torch.empty_like(head)
    se.se_rotary(head, None, pos, freqs, want)
    assert torch.equal(rows, want)
