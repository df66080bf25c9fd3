"""Paged attention, block-sparse partials and combine on another stream than the current one: what
they make does not take the place of memory that the current stream still reads."""
import numpy as np
import pytest
import torch

from paged_kv_cache_231_gb300 import binding as B

from .step_util import DEV, i32

pytestmark = pytest.mark.gpu


def _attention():
    gen = torch.Generator()
    gen.manual_seed(2)
    new = lambda *s: torch.randn(s, generator=gen).half().to(DEV)  # noqa: E731
    T = 2048
    table = i32(np.arange(T // 16)[None])
    a = [new(T, 1024), new(T, 256), new(T, 256), new(T // 16, 16, 4, 64), new(T // 16, 16, 4, 64),
         i32([0, T]), i32([0]), table]
    return lambda **kw: [B.pkv_paged_attention(*a, num_heads=16, kv_num_heads=4, **kw)]


def _combine():
    gen = torch.Generator()
    gen.manual_seed(3)
    o = torch.randn((4 * 16384, 64), generator=gen).to(DEV)
    m, l = (torch.rand(4 * 16384, generator=gen).to(DEV) + 0.5 for _ in range(2))
    return lambda **kw: [B.pkv_combine_partials(o, m, l, num_segments=16384, lanes=1,
                                                uniform_count=4, **kw)[0]]


def _partials():
    gen = torch.Generator()
    gen.manual_seed(4)
    new = lambda *s: torch.randn(s, generator=gen).to(DEV)  # noqa: E731
    n, edges = 64, 4096
    q, k, v = new(n, 8, 64), new(40, 2, 16, 64), new(40, 2, 16, 64)
    rng = np.random.default_rng(4)
    # query, kv head, block, sequence, keys of the block
    meta = i32(np.stack([rng.integers(0, top, edges) for top in (n, 2, 5, 2)] +
                        [np.full(edges, 64)], 1))
    table = i32(rng.permutation(40).reshape(2, 20))
    return lambda **kw: list(B.pkv_sparse_attention_partials(
        q, k, v, meta, table, qhead=4, block_size=64, page_size=16, pages_per_block=4,
        softmax_scale=0.125, **kw))


@pytest.mark.parametrize("make", [_attention, _combine, _partials])
def test_memory_that_the_current_stream_still_reads(make):
    call, side = make(), torch.cuda.Stream()
    out = call()
    torch.cuda.synchronize()
    want = [t.clone() for t in out]
    like = max(out, key=lambda t: t.numel() * t.element_size())
    for _ in range(3):
        freed = [torch.full_like(like, 7) for _ in range(6)]
        kept = [torch.empty_like(t) for t in freed]
        torch.cuda.synchronize()
        torch.cuda._sleep(40_000_000)
        for k, t in zip(kept, freed):
            k.copy_(t)
        del freed, t
        got = call(stream=side)
        side.synchronize()
        torch.cuda.synchronize()
        assert all(bool((k == 7).all()) for k in kept)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
