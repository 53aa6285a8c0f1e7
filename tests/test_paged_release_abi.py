"""Host-side checks of se_block_tables_release_ex: bad arguments are refused before any CUDA call (fake pointers,
never dereferenced)."""
import pytest

INVALID, UNSUPPORTED = 1, 2
FAKE = 0x7f0000000000

ARGS = ["free_pages", "pool_state", "num_pages", "block_table", "bt_stride", "seq_lens", "keep_lens", "batch",
        "seq_lens_after"]


@pytest.mark.parametrize("over,expect", [
    ({"batch": -1}, INVALID), ({"num_pages": -1}, INVALID), ({"bt_stride": 0}, INVALID),
    ({"free_pages": None}, INVALID), ({"pool_state": None}, INVALID), ({"block_table": None}, INVALID),
    ({"seq_lens": None}, INVALID), ({"keep_lens": FAKE + 4}, INVALID), ({"seq_lens_after": None}, INVALID),
    ({"seq_lens_after": FAKE + 4}, INVALID), ({"batch": 16385}, UNSUPPORTED), ({"num_pages": 1 << 27}, UNSUPPORTED),
    ({"batch": 0}, 0), ({"batch": 0, "seq_lens": None, "seq_lens_after": None}, 0),
])
def test_release_ex_refuses(se_lib, over, expect):
    a = dict.fromkeys(ARGS, FAKE)
    a.update(num_pages=64, bt_stride=8, batch=2)
    a.update(over)
    assert se_lib.se_block_tables_release_ex(*[a[n] for n in ARGS], None) == expect
    if expect:
        assert b"se_block_tables_release_ex" in se_lib.se_last_error_detail()
