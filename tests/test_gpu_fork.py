"""GPU parity of pkv_paged_fork."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as orc
from paged_kv_cache_231_gb300 import binding as B

from .step_util import DEV, i32

pytestmark = pytest.mark.gpu


class Case:
    """Rows of random lengths with random parents; caches of several widths and types."""

    def __init__(self, seed, rows, *, block_size=8, max_past=60, spare=20, layers=2, width=32,
                 parents=None, past=None, extra_columns=1):
        rng = np.random.default_rng(seed)
        self.bs = block_size
        self.past = rng.integers(0, max_past + 1, rows) if past is None else np.array(past)
        need = [-(-int(n) // block_size) for n in self.past]
        self.nb = max(1, sum(need) + spare)
        ids = rng.permutation(self.nb)
        self.table = rng.integers(-9, self.nb + 9, (rows, max(need) + extra_columns))
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.parents = (rng.integers(-1, rows, rows) if parents is None else np.array(parents))
        new = lambda dt, w: torch.randint(-9999, 9999, (self.nb, block_size, w)).to(dt)  # noqa: E731
        self.caches = [new(torch.float16, width) for _ in range(2 * layers)]
        self.caches += [new(torch.float32, 4), new(torch.uint8, 48)] if layers else []

    def check(self, status=None):
        caches = [c.to(DEV) for c in self.caches]
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        sizes = {} if caches else dict(num_blocks=self.nb, block_size=self.bs)
        args = [i32(self.parents), i32(self.past), i32(self.table)]
        past, table, free = B.pkv_paged_fork(*args, caches, device_status=st, **sizes)
        torch.cuda.synchronize()
        want = orc.fork(self.parents, self.past, self.table, [c.numpy() for c in self.caches],
                        num_blocks=self.nb, block_size=self.bs)
        assert past.tolist() == want[0]
        assert (table.cpu().numpy() == want[1]).all()
        assert free.item() == want[2]
        for got, ref in zip(caches, want[3]):
            assert np.array_equal(got.cpu().numpy(), ref)
        assert st.item() == (want[4] if status is None else status) == want[4]
        for t, x in zip(args, (self.parents, self.past, self.table)):
            assert (t.cpu().numpy() == x).all()
        return past, table, free


@pytest.mark.parametrize("rows", [1, 2, 3, 17, 64, 1030])
@pytest.mark.parametrize("block_size", [1, 8, 16, 24])
def test_random_parents(rows, block_size):
    for seed in range(3):
        Case(seed, rows, block_size=block_size, spare=rows).check()


@pytest.mark.parametrize("spare", [0, 1, 5])
def test_pool_too_small(spare):
    parents = [0] * 12
    c = Case(1, 12, past=[13] + [0] * 11, parents=parents, spare=spare)
    c.check(status=B.DEV_NO_BLOCKS)
    Case(2, 12, past=[16] + [0] * 11, parents=parents, spare=spare).check(status=0)


def test_what_goes_is_given_back():
    # the only free blocks are those that replaced rows leave
    c = Case(3, 6, past=[13, 20, 30, 7, 9, 40], parents=[0, 0, 0, -1, 4, 4], spare=0)
    past, _, free = c.check(status=0)
    assert past.tolist() == [13, 13, 13, 0, 9, 9] and free.item() > 0


def test_all_stay_and_all_go():
    Case(4, 30, parents=range(30)).check(status=0)
    _, table, free = Case(5, 30, parents=[-1] * 30).check(status=0)
    assert (table == -1).all() and free.item() == Case(5, 30).nb
    Case(6, 30, parents=list(range(1, 30)) + [0]).check(status=0)      # all change places


def test_bad_rows():
    c = Case(7, 8, past=[13, 5, 9, 6, 8, 0, 1, 60], parents=[0, 1, 8, 3, 0, 2 ** 31 - 1, -2 ** 31, 7])
    c.check(status=B.DEV_BAD_SEQUENCE)
    c.past[1] = -3
    c.check(status=B.DEV_BAD_SEQUENCE)
    c.parents = np.array([0, 0, 3, 3, 3, 7, 7, 7])
    c.past[3] = 10 ** 6
    c.check(status=B.DEV_BAD_BLOCK)


def test_entries_outside_the_pool():
    c = Case(8, 5, past=[20, 20, 20, 20, 20], parents=[0, 0, 1, 2, 2])
    c.table[0, 1] = -1          # a hole inside
    c.check(status=0)
    c.table[1, 2] = -1          # the partly filled one
    c.table[2, 0] = c.nb + 3
    c.check(status=B.DEV_BAD_BLOCK)
    c.table[2, 0] = 0
    c.table[2, 2] = -4
    c.check(status=B.DEV_BAD_BLOCK)


def test_shared_blocks():
    c = Case(9, 4, past=[30, 30, 30, 30], parents=[1, 1, 3, 3])
    c.table[1, :3] = c.table[0, :3]
    c.table[3] = c.table[2]     # a partly filled block that two rows share already
    c.check(status=0)


def test_tables_only_and_one_row():
    Case(10, 9, layers=0).check()
    Case(11, 1, past=[5], parents=[0]).check(status=0)


def test_wide_rows_and_long_tables():
    Case(12, 40, block_size=64, width=1024, layers=1, max_past=700).check()
    Case(13, 2000, block_size=4, width=8, layers=1, max_past=900, spare=500).check()


def test_twice_and_in_a_graph():
    c = Case(14, 12, spare=30)
    caches = [x.to(DEV) for x in c.caches]
    args = [i32(c.parents), i32(c.past), i32(c.table)]
    outs = dict(new_past_seqlens=torch.zeros(12, dtype=torch.int32, device=DEV),
                new_block_table=torch.zeros_like(args[2]),
                free_blocks=torch.zeros(1, dtype=torch.int32, device=DEV))
    B.pkv_paged_fork(*args, caches, **outs)
    torch.cuda.synchronize()
    want = [x.clone() for x in (*outs.values(), *caches)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.pkv_paged_fork(*args, caches, **outs)
    for _ in range(2):
        for x in outs.values():
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (*outs.values(), *caches)))
    s = torch.cuda.Stream()
    got = B.pkv_paged_fork(*args, caches, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
