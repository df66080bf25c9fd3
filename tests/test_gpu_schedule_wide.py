"""pkv_paged_schedule of rows as wide as a table may be."""
import pytest
import torch

from paged_kv_cache_231_gb300 import binding as B

from .step_util import DEV, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("columns", [2 ** 31 - 17, 2 ** 31 - 128, 2 ** 30 + 1])
def test_widest_row(columns):
    # blocks of one token: three are held, so two new ones are the lowest of the others
    table = torch.full((1, columns), 7, dtype=torch.int32, device=DEV)
    table[0, :3] = i32([3, 1, 0])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    cu, slots, pos, total, free = B.pkv_paged_schedule(
        i32([3]), i32([2]), table, num_blocks=8, block_size=1, num_tokens=2, device_status=status)
    torch.cuda.synchronize()
    assert cu.tolist() == [0, 2] and pos.tolist() == [3, 4] and total.tolist() == [5]
    assert slots.tolist() == [2, 4] and free.item() == 3 and status.item() == 0
    assert table[0, :6].tolist() == [3, 1, 0, 2, 4, 7]
