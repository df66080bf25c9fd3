"""Calls on another stream than the current one: what they make does not take the place of memory
that the current stream still reads, and in a capture it is the graph's."""
import pytest
import torch

from paged_kv_cache_231_gb300 import binding as B

from .step_util import DEV, CrossCase, i32

pytestmark = pytest.mark.gpu
ROWS = 2048


class Call:
    """One of the three operators; `like` has the size of the largest tensor that it makes."""

    def __init__(self, name):
        gen = torch.Generator()
        gen.manual_seed(1)
        new = lambda *s: torch.randn(s, generator=gen).half().to(DEV)  # noqa: E731
        self.name, self.kw = name, dict(num_heads=16, kv_num_heads=4)
        if name == "cross":
            c = CrossCase(90, [ROWS - 300, 300], [700, 2000], num_heads=16, kv_heads=4,
                          head_size=64, block_size=16)
            self.a = [c.q.to(DEV), c.k.to(DEV), c.v.to(DEV), i32(c.cu), i32(c.nk), i32(c.table)]
            self.f = B.pkv_cross_attention
        elif name == "append":
            self.a = [new(ROWS, 1024), new(ROWS, 256), new(ROWS, 256), new(200, 16, 4, 64),
                      new(200, 16, 4, 64), i32(range(ROWS)), None]
            self.f = B.pkv_paged_append_rotary_axes
        else:
            # long slot maps: tensors of 4 MB each
            self.a = [i32([5, 0]), i32([1 << 20, 9]), i32([[-1] * 40000] * 2)]
            self.a[2][0, 0] = 3
            self.kw = dict(num_blocks=40000, block_size=32, num_tokens=1 << 20)
            self.f = B.pkv_paged_schedule
        out = self()
        torch.cuda.synchronize()
        self.want = [t.clone() for t in out]
        self.like = max(out, key=lambda t: t.numel() * t.element_size())

    def __call__(self, **kw):
        out = self.f(*self.a, **self.kw, **kw)
        return list(out) if isinstance(out, tuple) else [out]

    def same(self, got):
        return all(torch.equal(x, y) for x, y in zip(got, self.want))


@pytest.mark.parametrize("name", ["schedule", "append", "cross"])
def test_memory_that_the_current_stream_still_reads(name):
    call, side = Call(name), torch.cuda.Stream()
    for _ in range(3):
        freed = [torch.full_like(call.like, 7) for _ in range(6)]
        kept = [torch.empty_like(t) for t in freed]
        torch.cuda.synchronize()
        torch.cuda._sleep(40_000_000)              # the current stream is behind
        for k, t in zip(kept, freed):
            k.copy_(t)
        del freed, t
        got = call(stream=side)                    # runs at once
        side.synchronize()
        torch.cuda.synchronize()
        assert all(bool((k == 7).all()) for k in kept)
        assert call.same(got)


@pytest.mark.parametrize("name", ["schedule", "append", "cross"])
def test_captured_on_a_forked_stream(name):
    call, side = Call(name), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        out = call(stream=side)
        here.wait_stream(side)
        copies = [t.clone() for t in out]
    for _ in range(3):
        for t in out + copies:
            t.zero_()
        junk = [torch.full_like(call.like, 9) for _ in range(8)]
        call(stream=side)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert call.same(out) and call.same(copies)
        assert all(bool((j == 9).all()) for j in junk)
