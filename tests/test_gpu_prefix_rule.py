"""When pkv_paged_prefix_attention shares: what that saves has to outweigh what the kernels cost that
would run. Told by the bits, which are those of the call that shares whatever it can, or others."""
import pytest
import torch

from paged_kv_cache_231_gb300 import binding as B

from .cache_util import CausalCase

pytestmark = pytest.mark.gpu


# query rows, keys of their own, shared keys, columns of the table, whether the longest sequence is
# named; saved, by the plan's count for 152 SMs, in us
@pytest.mark.parametrize("nq,own,keys,columns,named,shares", [
    # short keys of their own: beside the shared keys' tiles, 13 us are enough
    ([1] * 32, [16] * 32, 1536, None, True, True),                # 26.6
    ([1] * 64, [16] * 64, 512, 64, True, True),               # 17.4
    # the table's 34 blocks bound what can be saved: 64 * 544 * 8 * 128 * 4 / 7300 ns = 19.5 us,
    # less than the 24 us that sharing costs a call that need not look
    ([1] * 64, [16] * 64, 512, None, True, False),
    # one has many: an even share for every warp behind the tiles, 19 us are needed
    ([1] * 32, [3000] + [16] * 31, 768, None, True, False),   # 13.2
    ([1] * 32, [6000] + [16] * 31, 960, None, True, False),   # 16.6
    ([1] * 32, [3000] + [16] * 31, 2048, None, True, True),   # 35.6
    # tiles are launched for the keys of their own as well, 19 us
    ([1] * 32, [16] * 32, 960, None, False, False),           # 16.6
    ([1] * 32, [16] * 32, 1280, None, False, True),           # 22.2
    ([200, 150], [0, 7], 1024, None, True, False),            # prompts that fill tiles
])
def test_shares_where_that_saves_more(nq, own, keys, columns, named, shares):
    c = CausalCase(1, nq, [keys + x for x in own], groups=[(len(nq), keys)], num_heads=32,
                   kv_heads=8, head_size=128, max_blocks=columns)
    bits = []
    for mode in (0, 1):
        B.pkv_testing_prefix_sharing(mode)
        try:
            out, lse, status = c.gpu(prefix=True, max_query_len=max(nq) if named else 0)
        finally:
            B.pkv_testing_prefix_sharing()
        assert status == 0
        bits.append((out, lse))
    same = torch.equal(bits[0][0], bits[1][0]) and torch.equal(bits[0][1], bits[1][1])
    assert same == shares
    assert torch.allclose(bits[0][1], bits[1][1], atol=1e-4)
