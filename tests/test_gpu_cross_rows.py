"""Cross attention over cumulative lengths that do not ascend: the sequences that are bad get
nothing, the rows of the others stay theirs, whatever stands around them, and equal calls give
equal bits."""
import numpy as np
import pytest
import torch

from .step_util import CrossCase

pytestmark = pytest.mark.gpu


def _check(c, cu, **kw):
    first, lse = c.check(cu=np.array(cu, np.int32), **kw)
    assert torch.isfinite(first.float()).all()
    for _ in range(5):
        out, again, _ = c.gpu(cu=np.array(cu, np.int32), **kw)
        assert torch.equal(out, first) and torch.equal(again, lse)


# cumulative lengths for T rows; at most one valid sequence claims a row
ORDERS = [lambda T: [0, T + 5, 2, T], lambda T: [5, 2, T], lambda T: [T - 2, 0, T - 2],
          lambda T: [0, 1, T, 0, -4, 3], lambda T: [T, 0, T // 2, 3, T + 1, T // 2, T],
          lambda T: [2 ** 31 - 1, -2 ** 31, 1, T, 0, 1], lambda T: [T] + [0] * 40 + [T, 0]]


@pytest.mark.parametrize("order", range(len(ORDERS)))
@pytest.mark.parametrize("rows,max_blocks,max_query_len", [
    (8, 8, 8),          # a block for each sequence and kv head
    (8, 8192, 8),       # even shares of all steps
    (200, 8, 0),        # tiles
    (200, 300, 0)], ids=["small", "shares", "tiles", "long tiles"])
def test_descending_cumulative_lengths(order, rows, max_blocks, max_query_len):
    cu = ORDERS[order](rows)
    batch = len(cu) - 1
    keys = [50, 60, 70, 3, 90, 17, 1, 33]
    c = CrossCase(60 + order, [rows // batch] * batch, [keys[b % 8] for b in range(batch)],
                  num_heads=4, kv_heads=2, head_size=64, block_size=16, max_blocks=max_blocks,
                  pad=rows - rows // batch * batch)
    _check(c, cu, max_query_len=max_query_len)


@pytest.mark.parametrize("rows,max_query_len", [(8, 8), (300, 0)], ids=["few", "tiles"])
def test_a_sequence_without_states_beside_one_that_holds_the_row(rows, max_query_len):
    # both claim the rows: the one with states writes them, the other has nothing to write
    c = CrossCase(70, [2, 2, 2, 2], [40, 50, 60, 70], num_heads=4, kv_heads=2, head_size=128,
                  block_size=16, pad=rows - 8)
    cu, nk = [0, rows, 1, rows], [0, 50, 60]
    c.table, c.nk = c.table[:3], nk
    out, lse = c.check(cu=np.array(cu, np.int32), max_query_len=max_query_len)
    assert torch.isfinite(lse[1:]).all() and torch.isneginf(lse[0]).all()


def test_more_sequences_than_one_scan():
    # the valid sequence stands among 3000 of which every other descends
    cu = np.zeros(3001, np.int32)
    cu[1::2] = 7
    cu[1500:1502] = 1, 6
    c = CrossCase(71, [0] * 2999 + [8], [1] * 3000, num_heads=2, kv_heads=1, head_size=64,
                  block_size=16)
    nk = [0] * 3000
    nk[1500] = 1
    c.nk = nk
    _check(c, cu)
