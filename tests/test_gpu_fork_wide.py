"""pkv_paged_fork of rows as wide as a table may be."""
import pytest
import torch

from paged_kv_cache_231_gb300 import binding as B

from .step_util import DEV, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("columns", [2 ** 31 - 17, 2 ** 31 - 128, 2 ** 30 + 1])
def test_widest_row(columns):
    # blocks of one token: the entries of a row are counted up to 2^31 - 17
    table = torch.full((1, columns), 7, dtype=torch.int32, device=DEV)
    table[0, :4] = i32([3, 1, 0, 2])
    new = torch.full_like(table, 5)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    past, got, free = B.pkv_paged_fork(i32([0]), i32([3]), table, num_blocks=8, block_size=1,
                                       new_block_table=new, device_status=status)
    torch.cuda.synchronize()
    assert got is new and past.tolist() == [3] and free.item() == 5 and status.item() == 0
    assert got[0, :3].tolist() == [3, 1, 0]
    for at in range(3, columns, 1 << 28):
        assert (got[0, at:at + (1 << 28)] == -1).all()
    assert (table[0, 4:100] == 7).all() and (table[0, -100:] == 7).all()
