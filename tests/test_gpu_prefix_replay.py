"""One captured prefix attention, replayed with other lengths, groups and shared keys in the same
arrays: what its plan wrote the last time must not be seen again."""
import numpy as np
import pytest
import torch

from paged_kv_cache_231_gb300 import binding as B

from .cache_util import CausalCase
from .step_util import DEV, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["whatever can be", "by the rule"], autouse=True)
def sharing(request):
    B.pkv_testing_prefix_sharing(1 if request.param == "whatever can be" else 0)
    yield
    B.pkv_testing_prefix_sharing()


# (query rows of each sequence, tokens taken from its past, group offsets, shared keys)
FEW = [([1] * 12, [0] * 12, [0, 5, 12], [2048, 1024]),
       ([1] * 12, [7] * 12, [0, 5, 12], [512, 16]),
       ([1] * 12, [0] * 12, [0, 1, 2], [2048, 2048]),
       ([0] * 6 + [1] * 6, [0] * 12, [5, 6, 12], [0, 1000]),
       ([1] * 12, [0] * 12, [12, 3, 0], [2048, 1024]),     # descending: nothing is shared
       ([1] * 12, [0] * 12, [0, 2, 4], [2000, 1])]
MANY = [([40, 1, 0, 90, 3, 70], [0] * 6, [0, 3, 6], [2048, 1024]),
        ([1, 90, 60, 0, 50, 3], [100] * 6, [0, 3, 6], [640, 512]),
        ([34] * 6, [0] * 6, [0, 2, 4], [2048, 0]),
        ([0, 0, 204, 0, 0, 0], [0] * 6, [2, 3, 6], [2048, 2048]),
        ([40, 1, 0, 90, 3, 70], [0] * 6, [0, 7, 6], [2048, 1024]),
        ([2] * 5 + [194], [9] * 6, [0, 3, 6], [2048, 1024])]


@pytest.mark.parametrize("calls", [FEW, MANY], ids=["few", "many"])
@pytest.mark.parametrize("head_size,dtype,heads,kv", [(128, "bf16", 8, 2), (64, "f16", 4, 4)])
def test_replayed_with_other_lengths(calls, head_size, dtype, heads, kv):
    n, most = len(calls[0][0]), max(max(c[0]) for c in calls)
    past = [2048 + 30 * b for b in range(n)]
    # every sequence may take the most rows; the groups of the first call have their blocks
    # in common, and so have all groups that lie inside them
    offsets, shared = calls[0][2:]
    c = CausalCase(1, [most] * n, past, head_size=head_size, dtype=dtype, num_heads=heads,
                   kv_heads=kv, groups=[(b - a, s) for a, b, s in
                                        zip(offsets, offsets[1:], shared)])
    T = max(sum(x[0]) for x in calls)
    q = c.q[:T].to(DEV)
    k, v, table = c.k.to(DEV), c.v.to(DEV), i32(c.table)
    kw = dict(num_heads=heads, kv_num_heads=kv, max_query_len=most)

    def arrays(x):
        return [i32(np.concatenate([[0], np.cumsum(x[0])])),
                i32(np.array(past) - np.array(x[1])), i32(x[2]), i32(x[3])]

    cu, at, groups, keys = arrays(calls[0])
    out, lse = torch.empty_like(q), torch.empty((T, heads), device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.pkv_paged_prefix_attention(q, k, v, cu, at, table, groups, keys, output=out, lse=lse,
                                     device_status=status, **kw)
    for x in calls + calls[::-1] + calls:
        new = arrays(x)
        for old, y in zip((cu, at, groups, keys), new):
            old.copy_(y)
        out.fill_(float("nan"))
        status.zero_()
        g.replay()
        torch.cuda.synchronize()
        got, got_lse, flags = out.cpu(), lse.cpu(), int(status.item())
        want_lse = torch.empty_like(lse)
        want_status = torch.zeros_like(status)
        want = B.pkv_paged_prefix_attention(q, k, v, new[0], new[1], table, new[2], new[3],
                                            lse=want_lse, device_status=want_status, **kw)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.cpu().view(torch.int16))
        assert torch.equal(got_lse, want_lse.cpu()) and flags == int(want_status.item())
        assert not torch.isnan(got).any()
        wrong = any(b < a or not 0 <= a <= n or b > n for a, b in zip(x[2], x[2][1:]))
        assert flags == (B.DEV_BAD_SEQUENCE if wrong else 0)
