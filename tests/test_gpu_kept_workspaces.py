"""Kept workspaces that come and go (more streams than are kept for, releases between calls) while
calls are under way."""
import pytest
import torch

from paged_kv_cache_231_gb300 import binding as B

from .step_util import DEV, CrossCase, i32

pytestmark = pytest.mark.gpu


def test_more_streams_than_are_kept_for():
    c = CrossCase(97, [1, 70, 2, 1], [9000, 4000, 70, 12000], num_heads=8, kv_heads=2,
                  head_size=128, block_size=16)
    a = [c.q.to(DEV), c.k.to(DEV), c.v.to(DEV), i32(c.cu), i32(c.nk), i32(c.table)]
    kw = dict(num_heads=8, kv_num_heads=2)
    want = B.pkv_cross_attention(*a, **kw)
    streams = [torch.cuda.Stream() for _ in range(B._OWN_STREAMS + 3)]
    torch.cuda.synchronize()
    got = []
    for i in range(60):
        with torch.cuda.stream(streams[i * 3 % len(streams)]):
            got.append(B.pkv_cross_attention(*a, **kw))
        if i % 7 == 6:
            B.release_workspaces()
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    B.release_workspaces()
