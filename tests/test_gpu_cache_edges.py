"""The operators around the paged cache where calls go wrong: caches past 32-bit offsets, outputs at
odd 16 bytes, waits that give up, threads that share a stream, graphs beside eager calls."""
import threading

import numpy as np
import pytest
import torch

from paged_kv_cache_231_gb300 import binding as B

from .cache_util import CausalCase
from .step_util import DEV, i32
from .test_gpu_norm import Case as NormCase

pytestmark = pytest.mark.gpu


@pytest.fixture
def shared():
    B.pkv_testing_prefix_sharing(1)
    yield
    B.pkv_testing_prefix_sharing()


def far(c):
    """The case's cache behind 2^31 elements (2^32 bytes) of a larger one, and its table."""
    first = 2 ** 31 // (c.bs * c.hkv * c.d) + 5
    pools = []
    for x in (c.k, c.v):
        p = torch.empty((first + x.shape[0], *x.shape[1:]), dtype=c.t, device=DEV)
        p[first:] = x.to(DEV)
        pools.append(p)
    return pools, i32(np.where(c.table >= 0, c.table + first, -1))


@pytest.mark.parametrize("nq", [[1, 2], [140, 33]], ids=str)
@pytest.mark.parametrize("block_size", [16, 20])
def test_attention_past_32_bit_offsets(nq, block_size, shared):
    kw = dict(num_heads=8, kv_heads=8, head_size=128, block_size=block_size)
    c = CausalCase(1, nq, [300, 160], window=90, sinks=3, **kw)
    want, _, _ = c.gpu()
    (k, v), table = far(c)
    a = [c.q.to(DEV), k, v, i32(c.cu), i32(c.past), table]
    out = B.pkv_paged_window_attention(*a, num_heads=8, kv_num_heads=8, window=90, sinks=3)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want)
    del a, k, v, out
    c = CausalCase(2, nq, [300, 160], groups=[(2, 160)], **kw)
    want, _, _ = c.gpu(prefix=True)
    (k, v), table = far(c)
    out = B.pkv_paged_prefix_attention(c.q.to(DEV), k, v, i32(c.cu), i32(c.past), table,
                                       i32(c.groups), i32(c.shared), num_heads=8, kv_num_heads=8)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("head_size", [128, 72])
def test_append_past_32_bit_offsets(head_size):
    c = NormCase(3, 9, num_heads=8, kv_heads=8, head_size=head_size, rotary_dim=64, axes=1)
    want = [x.cpu() for x in c.check()]
    blocks = 2 ** 31 // (c.bs * c.hkv * c.d) + 7
    kc = torch.zeros((blocks, c.bs, c.hkv, c.d), dtype=c.t, device=DEV)
    vc, first = torch.zeros_like(kc), blocks - c.nb
    c.call(c.q.to(DEV), c.k.to(DEV), c.v.to(DEV), kc, vc, i32(c.slots + first * c.bs), i32(c.pos),
           None)
    torch.cuda.synchronize()
    row = lambda x: x.reshape(-1, c.hkv, c.d)[torch.from_numpy(c.slots).long()]  # noqa: E731
    assert torch.equal(row(kc[first:].cpu()), row(want[1]))
    assert torch.equal(row(vc[first:].cpu()), row(want[2]))


def test_fork_past_32_bit_offsets():
    bs, width = 64, 4096
    blocks = 2 ** 32 // (bs * width) + 40          # 4 GB of bytes
    c = torch.zeros((blocks, bs, width), dtype=torch.uint8, device=DEV)
    last = blocks - 30
    c[last] = torch.randint(0, 256, (bs, width), dtype=torch.uint8, device=DEV)
    # everything in front is held, so that the copy goes behind as well
    table = np.full((blocks // 1000 + 2, 1000), -1, np.int32)
    ids = np.arange(last)
    for b in range(len(table) - 2):
        table[b] = ids[b * 1000:(b + 1) * 1000][:1000] if (b + 1) * 1000 <= last else -1
    rest = ids[(last // 1000) * 1000:]
    full = last // 1000
    table[full:full + 1, :len(rest)] = rest
    rows = len(table)
    past = np.zeros(rows, np.int64)
    past[:full] = 1000 * bs
    past[full] = len(rest) * bs
    table = np.concatenate([table, np.full((2, 1000), -1, np.int32)])
    past = np.concatenate([past, [37, 0]])
    table[rows, 0] = last
    parents = np.arange(rows + 2)
    parents[rows + 1] = rows
    new_past, new_table, free = B.pkv_paged_fork(i32(parents), i32(past), i32(table), [c])
    torch.cuda.synchronize()
    to = int(new_table[rows + 1, 0])
    assert to == last + 1 and new_past[-1].item() == 37
    assert torch.equal(c[to, :37], c[last, :37]) and not c[to, 37:].any()


@pytest.mark.parametrize("head_size", [64, 128])
def test_output_at_16_bytes(head_size):
    c = CausalCase(4, [150, 1, 70], [10, 200, 0], window=60, sinks=2, head_size=head_size)
    want, _, _ = c.gpu()
    room = torch.zeros(c.q.numel() + 8, dtype=c.t, device=DEV)
    out = room[8:].view(c.q.shape)
    assert out.data_ptr() % 32 == 16
    B.pkv_paged_window_attention(*c.device(), num_heads=c.hq, kv_num_heads=c.hkv, window=60,
                                 sinks=2, output=out)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want) and not room[:8].any()


@pytest.mark.parametrize("head_size", [64, 128])
def test_waits_that_give_up(head_size, shared):
    c = CausalCase(5, [150, 1, 70], [64, 200, 64], groups=[(3, 64)], head_size=head_size)
    calls = (lambda: c.gpu(), lambda: c.gpu(prefix=True))
    want = [f() for f in calls]
    B.pkv_testing_wait_limit(4096, True)
    try:
        for f in calls:
            assert f()[2] == B.DEV_TIMEOUT
    finally:
        B.pkv_testing_wait_limit()
    for f, w in zip(calls, want):
        got = f()
        assert got[2] == 0 and torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])


def _case(seed):
    return CausalCase(seed, [1] * 20 + [60], [300 + 16 * i for i in range(20)] + [900],
                      groups=[(21, 288)], num_heads=8, kv_heads=2, head_size=128)


class Calls:
    """A window and a prefix attention, a fork and an append on data of their own."""

    def __init__(self, seed):
        c = self.c = _case(seed)
        self.a = c.device()
        self.more = [i32(c.groups), i32(c.shared)]
        self.parents = i32(np.random.default_rng(seed).integers(0, 21, 21))
        gen = torch.Generator()
        gen.manual_seed(seed)
        self.pool = torch.randn((c.k.shape[0] + 30, *c.k.shape[1:]), generator=gen).half().to(DEV)

    def __call__(self):
        kw = dict(num_heads=8, kv_num_heads=2)
        w = B.pkv_paged_window_attention(*self.a, window=100, sinks=4, **kw)
        p = B.pkv_paged_prefix_attention(*self.a, *self.more, **kw)
        f = B.pkv_paged_fork(self.parents, self.a[4], self.a[5], [self.pool])
        return [w, p, *f]


def test_threads_on_one_stream_and_on_two(shared):
    calls = [Calls(6), Calls(7)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    bad = []

    def work(c, expected, stream):
        with torch.cuda.stream(stream):
            got = [c() for _ in range(25)]
        torch.cuda.synchronize()
        bad.extend(1 for g in got for x, y in zip(g, expected)
                   if not torch.equal(x.view(torch.int16), y.view(torch.int16)))

    one = torch.cuda.Stream()
    for streams in ((one, one), (one, torch.cuda.Stream())):
        threads = [threading.Thread(target=work, args=x) for x in zip(calls, want, streams)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not bad


def test_two_graphs_and_eager_calls(shared):
    a, b = Calls(8), Calls(9)
    want = [a(), b()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append([c() for _ in range(2)])
        graphs.append(g)
    torch.cuda.synchronize()
    same = lambda x, y: all(torch.equal(p.view(torch.int16), q.view(torch.int16))  # noqa: E731
                            for p, q in zip(x, y))
    for _ in range(5):
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
        eager = [b() for _ in range(3)]
        torch.cuda.synchronize()
        assert all(same(x, want[0]) for x in outs[0]) and all(same(x, want[1]) for x in outs[1])
        assert all(same(x, want[1]) for x in eager)
