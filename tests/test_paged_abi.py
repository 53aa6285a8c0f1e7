"""Host-side checks of the page pool, the row store and the dense paged decode: bad arguments are
refused before any CUDA call (fake pointers, never dereferenced)."""
import ctypes

import pytest
import torch

import sparse_decode_attention_quest_gb300 as se

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
FAKE = 0x7f0000000000


def _kv(**over):
    f = dict(k=FAKE, v=FAKE + 4096, summary=None, num_pages=64, num_kv_heads=4, page_size=16,
             head_dim=128, head_dim_v=128, row_stride_k=128, row_stride_v=128)
    f.update(over)
    return se.SEPagedKV(**f)


EXTEND = ["free_pages", "pool_state", "num_pages", "block_table", "bt_stride", "seq_lens", "new_lens", "batch",
          "seq_lens_after", "token_start", "slot_map", "positions", "max_new_tokens"]


def _extend(lib, **over):
    a = dict.fromkeys(EXTEND, FAKE)
    a.update(num_pages=64, bt_stride=8, batch=2, max_new_tokens=32)
    a.update(over)
    return lib.se_block_tables_extend(*[a[n] for n in EXTEND], None)


@pytest.mark.parametrize("over,expect", [
    ({"batch": -1}, INVALID), ({"max_new_tokens": -1}, INVALID), ({"num_pages": -1}, INVALID),
    ({"bt_stride": 0}, INVALID), ({"free_pages": None}, INVALID), ({"pool_state": None}, INVALID),
    ({"block_table": None}, INVALID), ({"seq_lens": None}, INVALID), ({"new_lens": None}, INVALID),
    ({"seq_lens_after": None}, INVALID), ({"token_start": None}, INVALID), ({"slot_map": None}, INVALID),
    ({"slot_map": FAKE + 4}, INVALID), ({"positions": FAKE + 8}, INVALID), ({"seq_lens": FAKE + 4}, INVALID),
    ({"batch": 16385}, UNSUPPORTED), ({"num_pages": 1 << 27}, UNSUPPORTED), ({"bt_stride": 1 << 27}, UNSUPPORTED),
])
def test_extend_refuses(se_lib, over, expect):
    assert _extend(se_lib, **over) == expect
    assert b"se_block_tables_extend" in se_lib.se_last_error_detail()


RELEASE = ["free_pages", "pool_state", "num_pages", "block_table", "bt_stride", "seq_lens", "keep_lens", "batch"]


@pytest.mark.parametrize("over,expect", [
    ({"batch": -1}, INVALID), ({"num_pages": -1}, INVALID), ({"bt_stride": 0}, INVALID),
    ({"free_pages": None}, INVALID), ({"pool_state": None}, INVALID), ({"block_table": None}, INVALID),
    ({"seq_lens": None}, INVALID), ({"keep_lens": FAKE + 4}, INVALID), ({"batch": 16385}, UNSUPPORTED),
    ({"num_pages": 1 << 27}, UNSUPPORTED), ({"batch": 0}, 0), ({"batch": 0, "seq_lens": None}, 0),
])
def test_release_refuses(se_lib, over, expect):
    a = dict.fromkeys(RELEASE, FAKE)
    a.update(num_pages=64, bt_stride=8, batch=2)
    a.update(over)
    assert se_lib.se_block_tables_release(*[a[n] for n in RELEASE], None) == expect


@pytest.mark.parametrize("kv,over,expect", [
    (None, {}, INVALID), (_kv(k=None), {}, INVALID), (_kv(page_size=8), {}, INVALID),
    (_kv(head_dim=584, head_dim_v=584, row_stride_k=584, row_stride_v=584), {}, UNSUPPORTED),
    (_kv(), {"k_new": None}, INVALID), (_kv(), {"v_new": None}, INVALID), (_kv(), {"slot_map": None}, INVALID),
    (_kv(), {"num_tokens": -1}, INVALID), (_kv(), {"k_stride": 504}, INVALID), (_kv(), {"k_stride": 516}, INVALID),
    (_kv(), {"v_stride": 504}, INVALID), (_kv(), {"k_new": FAKE + 8}, INVALID), (_kv(), {"v_new": FAKE + 2}, INVALID),
    (_kv(), {"slot_map": FAKE + 4}, INVALID), (_kv(v=FAKE), {}, INVALID),  # latent: v_new must be NULL
    (_kv(), {"num_tokens": 0}, 0), (_kv(), {"num_tokens": 0, "k_new": None, "v_new": None, "slot_map": None}, 0),
])
def test_store_refuses(se_lib, kv, over, expect):
    a = dict(k_new=FAKE, k_stride=512, v_new=FAKE, v_stride=512, slot_map=FAKE, num_tokens=3)
    a.update(over)
    st = se_lib.se_paged_kv_store(None if kv is None else ctypes.byref(kv), a["k_new"], a["k_stride"], a["v_new"],
                                  a["v_stride"], a["slot_map"], a["num_tokens"], None)
    assert st == expect


LATENT = dict(v=FAKE, num_kv_heads=1, head_dim=576, head_dim_v=512, row_stride_k=576, row_stride_v=576)


@pytest.mark.parametrize("kv,over,expect", [
    (None, {}, INVALID), (_kv(v=None), {}, INVALID), (_kv(), {"batch": -1}, INVALID), (_kv(), {"hq": 30}, INVALID),
    (_kv(), {"hq": 0}, INVALID), (_kv(), {"hq": 4 * 65}, UNSUPPORTED),
    (_kv(head_dim=96, head_dim_v=96), {}, UNSUPPORTED), (_kv(head_dim_v=64), {}, UNSUPPORTED),
    (_kv(v=FAKE), {}, UNSUPPORTED),  # only the 576/512 latent cache shares its rows
    (_kv(**LATENT), {"hq": 8, "q_stride": 8 * 576}, UNSUPPORTED),
    (_kv(**LATENT), {"hq": 80, "q_stride": 80 * 576}, UNSUPPORTED),
    (_kv(**{**LATENT, "v": FAKE + 4096}), {"hq": 64, "q_stride": 64 * 576}, UNSUPPORTED),
    (_kv(), {"sink": -1}, INVALID), (_kv(), {"recent": -1}, INVALID), (_kv(), {"sink": 4}, INVALID),
    (_kv(), {"scale": float("inf")}, INVALID), (_kv(), {"q_stride": 4088}, INVALID), (_kv(), {"q_stride": 4100}, INVALID),
    (_kv(), {"bt_stride": 0}, INVALID), (_kv(), {"bt_stride": 1 << 27}, UNSUPPORTED),
    (_kv(), {"batch": 4097}, UNSUPPORTED), (_kv(), {"q": None}, INVALID), (_kv(), {"out": None}, INVALID),
    (_kv(), {"bt": None}, INVALID), (_kv(), {"lens": None}, INVALID), (_kv(), {"q": FAKE + 8}, INVALID),
    (_kv(), {"out": FAKE + 4}, INVALID), (_kv(), {"lse": FAKE + 4}, INVALID), (_kv(), {"ws": FAKE + 8}, INVALID),
    (_kv(), {"ws": None}, INVALID), (_kv(), {"ws_bytes": 15}, WORKSPACE), (_kv(), {"batch": 0, "q": None}, 0),
])
def test_decode_refuses(se_lib, kv, over, expect):
    a = dict(q=FAKE, q_stride=32 * 128, hq=32, bt=FAKE, bt_stride=8, lens=FAKE, batch=2, sink=0, recent=0, scale=0.1,
             out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 30)
    a.update(over)
    st = se_lib.se_paged_decode(None if kv is None else ctypes.byref(kv), a["q"], a["q_stride"], a["hq"], a["bt"],
                                a["bt_stride"], a["lens"], a["batch"], a["sink"], a["recent"], a["scale"], a["out"],
                                a["lse"], a["ws"], a["ws_bytes"], None)
    assert st == expect


def test_decode_workspace_size(se_lib):
    f = se_lib.se_paged_decode_workspace_size
    assert f(2, 32, 4, 128, 128) > 0 and f(2, 64, 1, 576, 512) > 0 and f(0, 8, 8, 64, 64) >= 0
    for bad in [(-1, 32, 4, 128, 128), (2, 30, 4, 128, 128), (2, 32, 4, 96, 96), (2, 32, 4, 128, 64),
                (2, 8, 1, 576, 512), (2, 65, 1, 128, 128)]:
        assert f(*bad) == 0


class _OnGpu(torch.Tensor):
    """A CPU tensor that says it is on cuda:0 (its pointer is not used)."""
    @staticmethod
    def __new__(cls, t):
        return torch.Tensor._make_subclass(cls, t)

    is_cuda = True

    def get_device(self):
        return 0


def test_binding_refuses_what_the_pointers_cannot_tell():
    bf16 = torch.bfloat16
    rows = torch.zeros(3, 4, 128, dtype=bf16)
    for t, dev, kind, text in [(rows, 0, ValueError, "CUDA tensor"), (_OnGpu(rows), 1, ValueError, "current device"),
                               (_OnGpu(rows.float()), 0, TypeError, "expected"), (3, 0, TypeError, "torch.Tensor"),
                               (_OnGpu(rows[:, :2]), 0, ValueError, "shape"), (_OnGpu(rows[0]), 0, ValueError, "shape"),
                               (_OnGpu(torch.zeros(3, 128, 4, dtype=bf16).transpose(1, 2)), 0, ValueError, "dense")]:
        with pytest.raises(kind, match=text):
            se._rows_ptr(t, 4, 128, bf16, "k_new", dev)
    # Rows a fused projection's width apart, and a single row of any stride, are fine.
    fused = torch.zeros(5, 12, 128, dtype=bf16)
    assert se._rows_ptr(_OnGpu(fused[:, 4:8]), 4, 128, bf16, "k", 0)[1] == 12 * 128
    assert se._rows_ptr(_OnGpu(fused[:1, 4:8]), 4, 128, bf16, "k", 0)[1] == 4 * 128
    slots = torch.zeros(4, 6, dtype=torch.int32)
    for t, n, kind, text in [(slots, 24, ValueError, "CUDA tensor"), (_OnGpu(slots), 23, ValueError, "elements"),
                             (_OnGpu(slots.long()), 24, TypeError, "expected"),
                             (_OnGpu(slots.t()), 24, ValueError, "contiguous")]:
        with pytest.raises(kind, match=text):
            se._vec(t, n, torch.int32, "slots", 0)
    with pytest.raises(ValueError, match="pages"):
        se._table(_OnGpu(slots[0]), "block_table", 0)
    assert se._table(_OnGpu(slots), "block_table", 0)[1:] == (4, 6)
