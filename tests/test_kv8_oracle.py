"""The oracle of the 8-bit cache against torch's e4m3 and against closed forms."""
import numpy as np
import pytest
import torch

import oracle.kv8 as k8


def test_codes_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(k8.VALUES, codes.view(torch.float8_e4m3fn).double().numpy())


def test_encode_rounds_as_torch_does():
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(20000, generator=g) * 10.0 ** torch.randint(-4, 2, (20000,), generator=g),
                   torch.arange(0, 448, 0.125), torch.arange(0, 1, 2.0 ** -11)]).clamp(-448, 448)
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(k8.encode(x.numpy()), want)
    assert k8.encode(np.nan) == k8.NAN_CODE


def test_scale_is_the_least_power_of_two():
    for a in [0.0, 1e-40, 448.0, 449.0, 3.5, 3.515625, 1.0, 3.3e38, 2.0 ** -91.3]:
        s = k8.scale_for(a)
        assert a <= 448 * s and (s == 2.0 ** -100 or a > 448 * s / 2) and np.log2(s) == round(np.log2(s))


def test_a_page_filled_token_by_token_is_the_page_filled_at_once():
    """But for values that a larger scale makes subnormal."""
    g = np.random.default_rng(2)
    rows = k8.to_bf16(g.standard_normal((16, 2, 64)) * np.exp2(g.integers(-3, 4, (16, 1, 1))))
    once, each = np.zeros((1, 2, 16, 64), np.uint8), np.zeros((1, 2, 16, 64), np.uint8)
    s1, s2 = np.zeros((1, 2), np.float32), np.zeros((1, 2), np.float32)
    k8.store(once, s1, rows, list(range(16)))
    for t in range(16):
        k8.store(each, s2, rows[t:t + 1], [t])
    np.testing.assert_array_equal(s1, s2)
    a, b = k8.values(once, s1), k8.values(each, s2)
    normal = np.abs(a) >= 2.0 ** -6 * s1[..., None, None]
    np.testing.assert_array_equal(a[normal], b[normal])
    assert (np.abs(a - b) <= 2.0 ** -9 * s1[..., None, None]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_keeps_products_of_equal_distances(interleaved):
    g = np.random.default_rng(3)
    q, k = g.standard_normal((1, 1, 64)), g.standard_normal((1, 1, 64))
    w, _ = k8.frequencies(64, 10000.0, "none")
    dot = lambda a, b: float((k8.rotary(q, [a], w, interleaved=interleaved) * k8.rotary(k, [b], w, interleaved=interleaved)).sum())
    assert abs(dot(5, 2) - dot(1003, 1000)) < 1e-9
    back = k8.rotary(k8.rotary(q, [77], w, interleaved=interleaved), [77], w, interleaved=interleaved, inverse=True)
    np.testing.assert_allclose(back, q, atol=1e-12)
