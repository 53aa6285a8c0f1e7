"""Page pool, block tables and slot maps on the GPU against a step-by-step simulation (whole numbers:
every comparison is exact)."""
import numpy as np
import pytest
import torch

import oracle.paged as op
import sparse_decode_attention_quest_gb300 as se

pytestmark = pytest.mark.gpu

UNUSED = -7  # what no call may change


class Case:
    """A pool and a table on the GPU beside the simulation's."""

    def __init__(self, dev, num_pages, width, batch, seed=0):
        g = np.random.default_rng(seed)
        self.pool = op.Pool(num_pages, g.permutation(num_pages))
        self.table = np.full((batch, width), UNUSED)
        self.lens = [0] * batch
        self.free = torch.tensor(self.pool.free, dtype=torch.int32, device=dev)
        self.state = torch.tensor([num_pages, 0, 0, 0], dtype=torch.int32, device=dev)
        self.t = torch.tensor(self.table, dtype=torch.int32, device=dev)
        self.l = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.dev = dev

    def extend(self, new, max_new, positions=True, in_place=True):
        self.table, after, start, slots, pos, err = op.extend(self.pool, self.table, self.lens, new, max_new)
        n = torch.tensor(new, dtype=torch.int32, device=self.dev)
        out = self.l if in_place else torch.full_like(self.l, UNUSED)
        ts = torch.full((len(new) + 1,), UNUSED, dtype=torch.int32, device=self.dev)
        sm = torch.full((max_new,), UNUSED, dtype=torch.int32, device=self.dev)
        ps = torch.full((max_new,), UNUSED, dtype=torch.int32, device=self.dev) if positions else None
        before = self.l.clone()
        se.se_block_tables_extend(self.free, self.state, self.t, self.l, n, out, ts, sm, ps)
        assert se.se_read_device_error(clear=True) == err
        assert self.t.cpu().numpy().tolist() == self.table.tolist()
        assert out.tolist() == after
        assert ts.tolist() == start
        assert sm.cpu().numpy().tolist() == slots.tolist()
        if positions:
            assert ps.cpu().numpy().tolist() == pos.tolist()
        if not in_place:
            assert torch.equal(self.l, before)
            self.l = out
        self.lens = after
        self.check_pool()
        return slots

    def release(self, keep=None):
        err = op.release(self.pool, self.table, self.lens, keep)
        k = None if keep is None else torch.tensor(keep, dtype=torch.int32, device=self.dev)
        t = self.t.clone()
        se.se_block_tables_release(self.free, self.state, self.t, self.l, k)
        assert se.se_read_device_error(clear=True) == err
        assert torch.equal(t, self.t)
        self.lens = [0] * len(self.lens) if keep is None else list(keep)
        self.l = torch.tensor(self.lens, dtype=torch.int32, device=self.dev)
        self.check_pool()

    def check_pool(self):
        assert self.state.tolist() == [len(self.pool.free), 0, 0, 0]
        assert self.free[:len(self.pool.free)].tolist() == [int(x) for x in self.pool.free]


@pytest.fixture(autouse=True)
def _no_device_errors(se_lib, cuda_device):
    se.se_read_device_error(clear=True)
    yield
    assert se.se_read_device_error(clear=True) == 0


@pytest.mark.parametrize("new", [[1], [16], [0], [15, 1, 17], [0, 0, 5, 0], [33, 0, 16, 1, 31, 48]])
@pytest.mark.parametrize("in_place", [False, True])
def test_steps_from_empty(cuda_device, new, in_place):
    c = Case(cuda_device, 64, 9, len(new))
    for k in range(3):
        c.extend(new, sum(new) + 3 * k, positions=k != 1, in_place=in_place)


@pytest.mark.parametrize("batch", [1, 31, 33, 511, 512, 513, 1025])
def test_batches(cuda_device, batch):
    g = np.random.default_rng(batch)
    c = Case(cuda_device, 6 * batch, 6, batch, seed=batch)
    for _ in range(3):
        new = g.integers(0, 30, batch).tolist()
        c.extend(new, sum(new) + 5)
    keep = [int(g.integers(0, n + 1)) for n in c.lens]
    c.release(keep)
    c.extend([1] * batch, batch)
    c.release()


def test_largest_batch(cuda_device):
    c = Case(cuda_device, 20000, 2, 16384, seed=6)
    g = np.random.default_rng(6)
    new = g.integers(0, 18, 16384).tolist()
    c.extend(new, sum(new))
    c.release([n // 2 for n in c.lens])
    with pytest.raises(se.SparseEngineError, match="16384"):
        z = lambda n: torch.zeros(n, dtype=torch.int32, device=cuda_device)
        se.se_block_tables_extend(c.free, c.state, z((16385, 2)), z(16385), z(16385), z(16385), z(16386), z(8))


@pytest.mark.parametrize("total", [2047, 2048, 2049, 70001])
def test_long_maps(cuda_device, total):
    """Maps that several CTAs fill, with a padded end."""
    new = [total // 3, 0, total - total // 3]
    c = Case(cuda_device, total // 16 + 8, total // 16 + 4, 3, seed=3)
    c.extend(new, total + 4099)
    c.extend([1, 1, 1], 3)
    c.release([5, 0, 17])


def test_a_release_undoes_an_extension(cuda_device):
    c = Case(cuda_device, 200, 20, 7, seed=4)
    c.extend([3, 40, 0, 16, 100, 1, 33], 300)
    before, free, state = list(c.lens), c.free.clone(), c.state.clone()
    c.extend([20, 1, 60, 16, 0, 15, 31], 200)
    c.release(before)
    assert torch.equal(free, c.free) and torch.equal(state, c.state)


@pytest.mark.parametrize("num_pages,new", [(0, [1]), (3, [16, 17, 16, 0, 1]), (3, [48, 1]), (4, [70, 1, 0])])
def test_too_few_pages(cuda_device, num_pages, new):
    """Requests are served in order until one finds too few pages; those that need none are served."""
    c = Case(cuda_device, num_pages, 8, len(new))
    c.extend(new, 200)


def test_a_request_behind_an_exhausted_pool_still_fills_its_page(cuda_device):
    c = Case(cuda_device, 2, 8, 3)
    c.extend([17, 0, 0], 20)
    c.extend([0, 1, 0], 20)          # no page left for the second
    c.extend([15, 4, 0], 20)         # the first still has room in its page


@pytest.mark.parametrize("lens,new,max_new", [
    ([0, -3, 5], [4, 4, 4], 20),                # a negative length
    ([0, 0, 0], [4, -4, 4], 20),
    ([0, 120, 0], [4, 9, 4], 20),               # one token more than the table holds
    ([0, 0, 0], [8, 8, 8], 20),                 # the last request's tokens do not fit the map
    ([0, 0, 0], [8, 100, 1], 20),
    ([0, 0, 0, 0], [2**31 - 1, 2**31 - 1, 2**31 - 1, 1], 20),  # sums beyond 32 bits
])
def test_lengths_out_of_bounds(cuda_device, lens, new, max_new):
    c = Case(cuda_device, 64, 8, len(lens))
    held = [max(0, min(n, 120)) for n in lens]
    c.extend(held, 128)
    c.lens = list(lens)
    c.l = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    c.extend(new, max_new)


def test_page_ids_out_of_range(cuda_device):
    c = Case(cuda_device, 16, 8, 2)
    c.extend([5, 20], 30)
    for bad in (16, -1, 2**31 - 1):
        c.table[0, 0] = bad
        c.t[0, 0] = bad
        c.extend([2, 1], 8)          # a table entry: its request's tokens get no slot
    c.pool.free[-1] = 99
    c.free[len(c.pool.free) - 1] = 99
    c.extend([16, 0], 16)            # a free page


def test_release_refuses_what_the_pool_cannot_hold(cuda_device):
    c = Case(cuda_device, 8, 8, 2)
    c.extend([40, 20], 60)
    c.release([41, 3])               # longer than the request: that request keeps its pages
    c.lens, c.l = [40, 3], torch.tensor([40, 3], dtype=torch.int32, device=cuda_device)
    c.release([40, 3])
    c.table[1] = 0
    c.t[1] = 0
    c.lens, c.l = [40, 128], torch.tensor([40, 128], dtype=torch.int32, device=cuda_device)
    c.release()                      # eleven pages into a pool of eight
    assert c.state.tolist()[0] == len(c.pool.free)


def test_empty_batch(cuda_device):
    c = Case(cuda_device, 4, 1, 0)
    c.extend([], 7)
    c.release()


def test_binding_checks_sizes(cuda_device):
    c = Case(cuda_device, 8, 2, 2)
    z = lambda n, d=torch.int32: torch.zeros(n, dtype=d, device=cuda_device)
    good = dict(free_pages=c.free, pool_state=c.state, block_table=c.t, seq_lens=c.l, new_lens=z(2),
                seq_lens_after=z(2), token_start=z(3), slot_map=z(4), positions=z(4))
    for name, bad in [("pool_state", z(3)), ("seq_lens", z(3)), ("new_lens", z(1)), ("token_start", z(2)),
                      ("positions", z(5)), ("seq_lens_after", z(3))]:
        with pytest.raises(ValueError):
            se.se_block_tables_extend(**{**good, name: bad})
    for name in good:
        with pytest.raises(TypeError):
            se.se_block_tables_extend(**{**good, name: good[name].float()})
    with pytest.raises(ValueError):
        se.se_block_tables_extend(**{**good, "slot_map": torch.zeros(4, dtype=torch.int32)})
