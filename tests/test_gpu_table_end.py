"""Causal attention of rows that stand behind the last key that the block table can name: the keys
in front of its end, the first ones among them, are still seen."""
import numpy as np
import pytest

from paged_kv_cache_231_gb300 import binding as B

from .cache_util import CausalCase

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nq,before,columns", [
    ([600], [284], 24),            # a tile that begins in front of the end, others behind it
    ([600, 40], [4, 0], 24),       # nearly all rows, and all rows of a sequence
    ([7, 1, 2], [0, 0, 1], 24),    # few rows
    ([300], [16], 1),              # a table of one block
], ids=str)
@pytest.mark.parametrize("window,sinks", [(30, 200), (1, 129), (30, 3), (64, 0), (16, 384)])
@pytest.mark.parametrize("block_size", [16, 20])
def test_first_keys_behind_the_end_of_the_table(nq, before, columns, window, sinks, block_size):
    end = columns * block_size     # the first row stands that many keys in front of it
    c = CausalCase(1, nq, [end - x for x in before], window=window, sinks=sinks,
                   block_size=block_size)
    c.table = np.ascontiguousarray(c.table[:, :columns])
    c.check(status=B.DEV_BAD_BLOCK)
