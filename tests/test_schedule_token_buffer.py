"""Token buffers that are too small: from the first row that they do not take on, no row that brings
tokens is granted any, however short it is."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as orc
from paged_kv_cache_231_gb300 import binding as B

CASES = [([3, 9, 2], 6, [0, 3, 3, 3]), ([5, 8, 2], 8, [0, 5, 5, 5]),
         ([7, 1, 1], 6, [0, 0, 0, 0]), ([2, 4, 0, 1], 6, [0, 2, 6, 6, 6])]


def _oracle(new, tokens):
    return orc.schedule([0] * len(new), new, np.full((len(new), 4), -1), num_blocks=20,
                        block_size=4, num_tokens=tokens)


@pytest.mark.parametrize("new,tokens,cu", CASES)
def test_oracle(new, tokens, cu):
    got = _oracle(new, tokens)
    assert got[0].tolist() == cu and got[-1] == orc.BAD_SEQUENCE


@pytest.mark.gpu
@pytest.mark.parametrize("new,tokens,cu", CASES)
def test_kernel(new, tokens, cu):
    i32 = dict(dtype=torch.int32, device="cuda")
    table, status = torch.full((len(new), 4), -1, **i32), torch.zeros(1, **i32)
    got = B.pkv_paged_schedule(torch.zeros(len(new), **i32), torch.tensor(new, **i32), table,
                               num_blocks=20, block_size=4, num_tokens=tokens,
                               device_status=status)
    ref = _oracle(new, tokens)
    for g, r in zip([*got, table, status], ref):
        assert g.flatten().tolist() == np.asarray(r).reshape(-1).tolist()
    assert got[0].tolist() == cu
