"""Cross attention with cumulative lengths from the ends of the 32-bit range: such sequences are
refused, whatever their difference wraps around to."""
import numpy as np
import pytest

from .step_util import CrossCase

pytestmark = pytest.mark.gpu
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("rows,max_blocks,max_query_len", [(8, 8, 8), (8, 8192, 8), (200, 8, 0)],
                         ids=["small", "shares", "tiles"])
@pytest.mark.parametrize("ends", [(HIGH, LOW), (HIGH, LOW + 5), (LOW, HIGH), (LOW, LOW + 3),
                                  (HIGH - 2, HIGH)], ids=str)
def test_lengths_whose_difference_does_not_fit(ends, rows, max_blocks, max_query_len):
    c = CrossCase(80, [rows, 0], [50, 60], num_heads=4, kv_heads=2, head_size=64, block_size=16,
                  max_blocks=max_blocks)
    c.check(cu=np.array([*ends, ends[1]], np.int64).astype(np.int32), max_query_len=max_query_len)
