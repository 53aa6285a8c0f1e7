"""Host-side checks of the rotary calls and the 8-bit cache's: bad arguments are refused before any CUDA call (fake
pointers, never dereferenced), and the frequencies, which are computed on the host."""
import ctypes
import math
import types
from decimal import Decimal, getcontext

import pytest
import torch

import sparse_decode_attention_quest_gb300 as se

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
FAKE = 0x7f0000000000


def _kv(**over):
    f = dict(k=FAKE, v=FAKE + 4096, k_scale=FAKE + 8192, v_scale=FAKE + 12288, num_pages=64, num_kv_heads=4,
             page_size=16, head_dim=128)
    f.update(over)
    return se.SEPagedKV8(**f)


BAD_VIEWS = [(None, INVALID), (_kv(k=None), INVALID), (_kv(v=None), INVALID), (_kv(k_scale=None), INVALID),
             (_kv(v_scale=None), INVALID), (_kv(k=FAKE + 8), INVALID), (_kv(v_scale=FAKE + 4), INVALID),
             (_kv(v=FAKE), INVALID), (_kv(v_scale=FAKE + 8192), INVALID), (_kv(page_size=8), INVALID),
             (_kv(num_pages=-1), INVALID), (_kv(num_kv_heads=0), INVALID), (_kv(head_dim=96), UNSUPPORTED),
             (_kv(head_dim=576), UNSUPPORTED), (_kv(num_pages=1 << 27), UNSUPPORTED)]


def _ref(kv):
    return None if kv is None else ctypes.byref(kv)


STORE = dict(k_new=FAKE, k_stride=512, v_new=FAKE, v_stride=512, slot_map=FAKE, num_tokens=3)


@pytest.mark.parametrize("kv,over,expect", [(kv, {}, e) for kv, e in BAD_VIEWS] + [
    (_kv(), {"k_new": None}, INVALID), (_kv(), {"v_new": None}, INVALID), (_kv(), {"slot_map": None}, INVALID),
    (_kv(), {"num_tokens": -1}, INVALID), (_kv(), {"k_stride": 504}, INVALID), (_kv(), {"k_stride": 516}, INVALID),
    (_kv(), {"v_stride": 504}, INVALID), (_kv(), {"v_stride": 513}, INVALID), (_kv(), {"k_new": FAKE + 8}, INVALID),
    (_kv(), {"v_new": FAKE + 2}, INVALID), (_kv(), {"slot_map": FAKE + 4}, INVALID),
    (_kv(), {"num_tokens": 0, "k_new": None, "v_new": None, "slot_map": None}, 0),
])
def test_store_refuses(se_lib, kv, over, expect):
    assert se_lib.se_paged_kv8_store(_ref(kv), *{**STORE, **over}.values(), None) == expect


LOAD = dict(block_table=FAKE, bt_stride=8, first=None, token_start=FAKE, batch=2, num_rows=20, k_out=FAKE, k_stride=512,
            v_out=FAKE, v_stride=512)


@pytest.mark.parametrize("kv,over,expect", [(kv, {}, e) for kv, e in BAD_VIEWS] + [
    (_kv(), {"block_table": None}, INVALID), (_kv(), {"token_start": None}, INVALID), (_kv(), {"k_out": None}, INVALID),
    (_kv(), {"v_out": None}, INVALID), (_kv(), {"bt_stride": 0}, INVALID), (_kv(), {"batch": -1}, INVALID),
    (_kv(), {"num_rows": -1}, INVALID), (_kv(), {"batch": 16385}, UNSUPPORTED), (_kv(), {"bt_stride": 1 << 27}, UNSUPPORTED),
    (_kv(), {"first": FAKE + 4}, INVALID), (_kv(), {"token_start": FAKE + 4}, INVALID), (_kv(), {"k_out": FAKE + 8}, INVALID),
    (_kv(), {"k_stride": 504}, INVALID), (_kv(), {"v_stride": 516}, INVALID), (_kv(), {"batch": 0, "k_out": None}, 0),
    (_kv(), {"num_rows": 0, "block_table": None}, 0),
])
def test_load_refuses(se_lib, kv, over, expect):
    assert se_lib.se_paged_kv8_load(_ref(kv), *{**LOAD, **over}.values(), None) == expect


DECODE = dict(q=FAKE, q_stride=32 * 128, hq=32, bt=FAKE, bt_stride=8, lens=FAKE, batch=2, sink=0, recent=0, scale=0.1,
              out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 30)


@pytest.mark.parametrize("kv,over,expect", [(kv, {}, e) for kv, e in BAD_VIEWS] + [
    (_kv(), {"batch": -1}, INVALID), (_kv(), {"hq": 30}, INVALID), (_kv(), {"hq": 0}, INVALID),
    (_kv(), {"hq": 4 * 65}, UNSUPPORTED), (_kv(), {"sink": -1}, INVALID), (_kv(), {"recent": -1}, INVALID),
    (_kv(), {"sink": 4}, INVALID), (_kv(), {"scale": float("inf")}, INVALID), (_kv(), {"scale": float("nan")}, INVALID),
    (_kv(), {"q_stride": 4088}, INVALID), (_kv(), {"q_stride": 4100}, INVALID), (_kv(), {"bt_stride": 0}, INVALID),
    (_kv(), {"bt_stride": 1 << 27}, UNSUPPORTED), (_kv(), {"batch": 4097}, UNSUPPORTED), (_kv(), {"q": None}, INVALID),
    (_kv(), {"out": None}, INVALID), (_kv(), {"bt": None}, INVALID), (_kv(), {"lens": None}, INVALID),
    (_kv(), {"q": FAKE + 8}, INVALID), (_kv(), {"out": FAKE + 4}, INVALID), (_kv(), {"lse": FAKE + 4}, INVALID),
    (_kv(), {"ws": FAKE + 8}, INVALID), (_kv(), {"ws": None}, INVALID), (_kv(), {"ws_bytes": 15}, WORKSPACE),
    (_kv(), {"batch": 0, "q": None}, 0),
])
def test_decode_refuses(se_lib, kv, over, expect):
    assert se_lib.se_paged_kv8_decode(_ref(kv), *{**DECODE, **over}.values(), None) == expect


def test_decode_workspace_size(se_lib):
    f = se_lib.se_paged_kv8_decode_workspace_size
    for h, d in [(1, 64), (4, 128), (8, 256)]:
        assert f(4096, 32, h, d) == f(1, 32, h, d) > 0
    for bad in [(-1, 32, 4, 128), (4097, 32, 4, 128), (2, 30, 4, 128), (2, 32, 4, 96), (2, 32, 4, 576), (2, 65, 1, 128),
                (2, 0, 1, 128), (2, 4, 0, 128)]:
        assert f(*bad) == 0


ROTARY = dict(q=FAKE, q_stride=1024, hq=8, k=FAKE + 4096, k_stride=256, hk=2, dim=128, offset=0, rot=128, flags=0,
              freqs=FAKE, amplitude=1.0, positions=FAKE, valid=None, tokens=3, q_out=FAKE, q_out_stride=1024,
              k_out=FAKE + 4096, k_out_stride=256)


@pytest.mark.parametrize("over,expect", [
    ({"q": None}, INVALID), ({"q_out": None}, INVALID), ({"k": None}, INVALID), ({"k_out": None}, INVALID),
    ({"hq": 0}, INVALID), ({"hk": 0}, INVALID),  # rows without heads
    ({"hq": -1}, INVALID), ({"hk": -1}, INVALID), ({"tokens": -1}, INVALID),
    ({"hq": 0, "hk": 0, "q": None, "k": None, "q_out": None, "k_out": None}, INVALID),
    ({"hq": 1023, "q_stride": 1 << 20, "q_out_stride": 1 << 20}, UNSUPPORTED),
    ({"dim": 0}, INVALID), ({"dim": 100}, INVALID), ({"dim": 584}, UNSUPPORTED), ({"rot": 0}, INVALID),
    ({"rot": 12}, INVALID), ({"rot": 136}, INVALID), ({"offset": 8}, INVALID), ({"offset": -8}, INVALID),
    ({"offset": 4, "rot": 64}, INVALID), ({"flags": 4}, INVALID), ({"amplitude": float("nan")}, INVALID),
    ({"freqs": None}, INVALID), ({"positions": None}, INVALID), ({"freqs": FAKE + 8}, INVALID),
    ({"positions": FAKE + 4}, INVALID), ({"valid": FAKE + 2}, INVALID), ({"q": FAKE + 8}, INVALID),
    ({"k_out": FAKE + 2}, INVALID), ({"q_stride": 1016}, INVALID), ({"q_stride": 1028}, INVALID),
    ({"k_out_stride": 248}, INVALID), ({"q_out_stride": 1032}, INVALID),  # in place with another stride
    ({"tokens": 0, "freqs": None}, 0),
])
def test_rotary_refuses(se_lib, over, expect):
    assert se_lib.se_rotary(*{**ROTARY, **over}.values(), None) == expect


@pytest.mark.parametrize("over", [
    dict(rotary_dim=0), dict(rotary_dim=7), dict(base=1.0), dict(base=float("inf")), dict(base=float("nan")),
    dict(factor=0.5), dict(factor=float("nan")), dict(scaling="yarn"), dict(scaling="yarn", original_len=-4)])
def test_frequencies_refuse(se_lib, over):
    with pytest.raises(se.SparseEngineError):
        se.se_rotary_frequencies(**{**dict(rotary_dim=64, factor=4.0), **over})


def test_frequencies_refuse_unknown_scalings(se_lib):
    with pytest.raises(ValueError, match="scaling"):
        se.se_rotary_frequencies(64, scaling="other")
    out = (ctypes.c_uint64 * 4)()
    amp = ctypes.c_float()
    assert se_lib.se_rotary_frequencies(8, 1e4, 4, 1.0, 0, out, ctypes.byref(amp)) == INVALID
    assert se_lib.se_rotary_frequencies(8, 1e4, 0, 1.0, 0, None, ctypes.byref(amp)) == INVALID
    assert se_lib.se_rotary_frequencies(8, 1e4, 0, 1.0, 0, out, None) == INVALID


@pytest.mark.parametrize("dim,base,scaling,factor,original", [
    (128, 1e4, "none", 1.0, 0), (64, 1e6, "linear", 4.0, 0), (96, 1e4, "ntk", 8.0, 0), (2, 1e4, "ntk", 8.0, 0),
    (128, 1e4, "yarn", 4.0, 4096), (72, 5e5, "yarn", 32.0, 8192)])
def test_frequencies(se_lib, dim, base, scaling, factor, original):
    """Against 40 digits. The power, its arguments and the quotients are off by a few steps of 2^-53 each: 16 of them."""
    getcontext().prec = 40
    pi = Decimal("3.141592653589793238462643383279502884197")
    got, amp = se.se_rotary_frequencies(dim, base, scaling, factor, original)
    assert got.dtype == torch.int64 and got.numel() == dim // 2
    b, s = Decimal(base), Decimal(factor)
    if scaling == "ntk" and dim > 2:
        b = b * (s.ln() * dim / (dim - 2)).exp()
    for i in range(dim // 2):
        w = (-2 * b.ln() * i / dim).exp()
        if scaling == "linear":
            w /= s
        if scaling == "yarn":
            g = min(Decimal(1), max(Decimal(0), (original * w / (2 * pi) - 1) / 31))
            w = w * g + w / s * (1 - g)
        want = w / (2 * pi) * 2 ** 64
        assert abs((int(got[i]) & (2 ** 64 - 1)) - want) <= want * 16 * Decimal(2) ** -53 + 1
    assert amp == pytest.approx(0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0, rel=1e-7)


def _on(index, *shape, dtype=torch.bfloat16):
    """What the binding looks at of a CUDA tensor on device ``index``."""
    class OnGpu(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return index

    return torch.Tensor._make_subclass(OnGpu, torch.zeros(*shape, dtype=torch.float32).to(dtype))


@pytest.fixture
def current(monkeypatch):
    """Current device 0 and a library whose calls succeed without running."""
    made = []
    ok = lambda name: lambda *a: made.append(name) or 0
    lib = types.SimpleNamespace(se_rotary=ok("rotary"), se_paged_kv8_store=ok("store"), se_paged_kv8_load=ok("load"),
                                se_paged_kv8_decode=ok("decode"))
    monkeypatch.setattr(se, "load_library", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return made


F8, I32 = torch.float8_e4m3fn, torch.int32


def _view8(index=0, **over):
    a = dict(k_cache=_on(index, 4, 2, 16, 64, dtype=F8), v_cache=_on(index, 4, 2, 16, 64, dtype=F8),
             k_scale=_on(index, 4, 2, dtype=torch.float32), v_scale=_on(index, 4, 2, dtype=torch.float32))
    return se.paged_kv8(**{**a, **over})


def test_views(se_lib):
    assert _view8().device == 0 and _view8().head_dim == 64
    for over, kind in [(dict(k_cache=_on(0, 4, 2, 16, 64)), TypeError), (dict(v_cache=_on(0, 4, 2, 16, 32, dtype=F8)), ValueError),
                       (dict(k_scale=_on(0, 4, 1, dtype=torch.float32)), ValueError), (dict(v_scale=_on(0, 4, 2)), TypeError),
                       (dict(k_cache=_on(0, 4, 2, 8, 64, dtype=F8)), ValueError), (dict(v_cache=None), TypeError),
                       (dict(k_scale=_on(1, 4, 2, dtype=torch.float32)), ValueError)]:
        with pytest.raises(kind):
            _view8(**over)


def test_another_device_and_other_views(current):
    rows, slots = _on(0, 3, 2, 64), _on(0, 3, dtype=I32)
    table, start = _on(0, 2, 3, dtype=I32), _on(0, 3, dtype=I32)
    calls = {
        "store": lambda kv: se.se_paged_kv8_store(kv, rows, rows, slots, stream=5),
        "load": lambda kv: se.se_paged_kv8_load(kv, table, start, rows, rows, stream=5),
        "decode": lambda kv: se.se_paged_kv8_decode(kv, _on(0, 2, 4, 64), table, _on(0, 2, dtype=I32), 0.1, _on(0, 2, 4, 64),
                                                    None, _on(0, 64, dtype=torch.uint8), stream=5)}
    for call in calls.values():
        call(_view8())
        with pytest.raises(ValueError, match="kv: is on cuda:1"):
            call(_view8(1))
        with pytest.raises(TypeError, match="8-bit"):
            call(se.SEPagedKV(FAKE, FAKE + 64, None, 4, 2, 16, 64, 64, 64, 64))
    assert current == list(calls)


def test_rotary_binding(current):
    pos, freqs = _on(0, 3, dtype=I32), _on(0, 8, dtype=torch.int64)
    q, k = _on(0, 3, 4, 64), _on(0, 3, 2, 64)
    se.se_rotary(q, k, pos, freqs, stream=5)
    se.se_rotary(q, None, pos, freqs, stream=5)
    se.se_rotary(None, k, pos, freqs, None, k, stream=5)
    assert current == ["rotary"] * 3
    for args, kind in [((None, None, pos, freqs), ValueError), ((q[:2], k, pos, freqs), ValueError),
                       ((q, _on(0, 3, 2, 128), pos, freqs), ValueError), ((q, k, pos, _on(0, 8, dtype=I32)), TypeError),
                       ((q, k, _on(0, 3), freqs), TypeError), ((q, k, _on(1, 3, dtype=I32), freqs), ValueError),
                       ((q, k, pos, freqs, q[:2]), ValueError), ((q, None, pos, freqs, None, k), ValueError),
                       ((q.float(), k, pos, freqs), TypeError), ((q[0], k, pos, freqs), ValueError)]:
        with pytest.raises(kind):
            se.se_rotary(*args, stream=5)
    with pytest.raises(ValueError, match="num_valid"):
        se.se_rotary(q, k, pos, freqs, num_valid=pos, stream=5)
    assert len(current) == 3
