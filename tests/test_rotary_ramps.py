"""The ramp of scaled rotary frequencies by pairs: on the host against its definition in 40 digits and at the pairs where
it begins and ends, and on the GPU as angles."""
import ctypes
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import oracle.kv8 as k8
import sparse_decode_attention_quest_gb300 as se

PI = Decimal("3.141592653589793238462643383279502884197")
# (rotary dim, base, factor, original length), and the pairs at which the ramp begins and ends, worked out by hand from
# dim ln(length / (2 pi turns)) / (2 ln base) with 32 turns and one: 20.94 and 45.03; 10.47 and 22.51; 23.60 and 39.65;
# 19.32 and 37.38; -1.60 (none: 0) and 1.41.
RAMPS = [((128, 1e4, 4.0, 4096), 20, 46), ((64, 1e4, 40.0, 4096), 10, 23), ((128, 1e6, 4.0, 32768), 23, 40),
         ((72, 1e3, 8.0, 8192), 19, 38), ((16, 1e4, 2.0, 32), 0, 2)]


def _turns(freqs):
    return [Decimal(int(f) & (2 ** 64 - 1)) / Decimal(2) ** 64 for f in freqs]


def _plain(dim, base):
    getcontext().prec = 40
    return [(-2 * Decimal(base).ln() * i / dim).exp() / (2 * PI) for i in range(dim // 2)]


@pytest.mark.parametrize("args,low,high", RAMPS)
def test_ends_of_the_ramp(se_lib, args, low, high):
    """Pairs up to the first end keep their frequencies, those from the second on have them divided, those between are
    mixed in equal steps. 16 steps of 2^-53 and half a step of 2^-64 for the power, its argument and the quotients."""
    dim, base, factor, original = args
    got, amp = se.se_rotary_frequencies(dim, base, "yarn_pairs", factor, original)
    assert amp == pytest.approx(0.1 * math.log(factor) + 1, rel=1e-7)
    for i, (f, w) in enumerate(zip(_turns(got), _plain(dim, base))):
        mixed = min(Decimal(1), max(Decimal(0), Decimal(i - low) / (high - low)))
        want = w * (1 - mixed) + w / Decimal(factor) * mixed
        assert abs(f - want) <= want * 16 * Decimal(2) ** -53 + Decimal(2) ** -64


def test_ends_that_meet(se_lib):
    """All pairs make more than 32 turns, or fewer than one: no ramp is left, and nothing is divided by zero."""
    for original, divided in ((2 ** 31 - 1, Decimal(1)), (6, Decimal(4))):
        got, _ = se.se_rotary_frequencies(16, 4.0, "yarn_pairs", 4.0, original)
        for f, w in list(zip(_turns(got), _plain(16, 4.0)))[1:]:
            assert abs(f - w / divided) <= w * 16 * Decimal(2) ** -53 + Decimal(2) ** -64


def test_the_two_ramps_differ(se_lib):
    """By tens of percent between their ends (the paper's ramp falls much faster), not at all in the outer pairs."""
    a, b = (np.array([float(x) for x in _turns(se.se_rotary_frequencies(128, 1e4, s, 4.0, 32768)[0])])
            for s in ("yarn", "yarn_pairs"))
    off = np.abs(a - b) / np.maximum(a, b)
    assert off[0] == off[-1] == 0 and 0.3 < off.max() < 0.75


def test_refusals(se_lib):
    out, amp = (ctypes.c_uint64 * 4)(), ctypes.c_float()
    call = lambda scaling, factor, original: se_lib.se_rotary_frequencies(8, 1e4, scaling, factor, original, out,
                                                                          ctypes.byref(amp))
    assert call(se.ROTARY_SCALINGS["yarn_pairs"], 4.0, 4096) == 0
    for bad in ((19, 4.0, 0), (19, 4.0, -1), (19, 0.5, 4096), (16, 4.0, 4096), (18, 4.0, 4096), (20, 4.0, 4096), (-1, 4.0, 4096)):
        assert call(*bad) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("scaling", [("none", 1.0, 0), ("ntk", 4.0, 0), ("yarn", 4.0, 32768), ("yarn_pairs", 4.0, 32768),
                                     ("yarn_pairs", 40.0, 4096)])
@pytest.mark.parametrize("base", [100.0, 5e5, 1e6, 1e8])
def test_rotation(cuda_device, base, scaling):
    """With D = |x0| + |x1|: angles within 2^-22 (32 bits of a turn, fp32) and 2^-49 of themselves (frequencies), cosine, sine,
    products and their difference 6 steps of 2^-23, then bf16."""
    positions = [0, 1, 77, 4095, 100000, 999999, 2 ** 31 - 1]
    x = torch.randn(len(positions), 3, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    freqs, amplitude = se.se_rotary_frequencies(128, base, *scaling)
    w, amp = k8.frequencies(128, base, *scaling)
    out = torch.empty_like(x, device=cuda_device)
    se.se_rotary(x.to(cuda_device), None, torch.tensor(positions, dtype=torch.int32, device=cuda_device),
                 freqs.to(cuda_device), out, amplitude=amplitude)
    src, got = x.double().numpy(), out.double().cpu().numpy()
    ref = k8.rotary(src, positions, w, amplitude=amp)
    far = 2.0 ** -49 * np.array(positions, dtype=np.float64)[:, None, None]
    tol = (2.0 ** -22 + 6 * 2.0 ** -23 + far) * amp * (np.abs(src) + np.abs(np.roll(src, 64, -1)))
    assert (np.abs(got - ref) <= tol + 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7)).all()
