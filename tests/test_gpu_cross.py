"""GPU parity of pkv_cross_attention against its definition in 64 bits."""
import threading

import numpy as np
import pytest
import torch

from paged_kv_cache_231_gb300 import binding as B

from .step_util import DEV, CrossCase, i32

pytestmark = pytest.mark.gpu
BOTH = pytest.mark.parametrize("dtype", ["f16", "bf16"])


@BOTH
@pytest.mark.parametrize("heads,kv,d,bs", [
    (4, 2, 64, 16), (8, 8, 128, 16), (16, 1, 128, 32), (6, 2, 64, 8), (5, 1, 128, 64),
    (4, 2, 128, 7), (2, 2, 64, 1), (8, 1, 64, 24), (32, 8, 128, 128)])
@pytest.mark.parametrize("nq,nk", [
    ([1], [1]), ([1, 1, 1], [0, 17, 400]), ([1] * 9, [5, 16, 31, 32, 33, 127, 128, 129, 1000]),
    ([2, 1, 3], [64, 0, 90])], ids=["one", "few", "edges", "drafts"])
def test_few_rows(heads, kv, d, bs, nq, nk, dtype):
    CrossCase(11, nq, nk, num_heads=heads, kv_heads=kv, head_size=d, block_size=bs,
              dtype=dtype).check()


@BOTH
@pytest.mark.parametrize("heads,kv,d,bs", [
    (4, 2, 64, 16), (4, 4, 128, 32), (16, 1, 128, 16), (6, 2, 64, 8), (5, 1, 128, 64),
    (4, 2, 128, 7), (2, 1, 64, 20), (8, 2, 128, 128), (3, 3, 64, 256)])
@pytest.mark.parametrize("nq,nk", [
    ([17], [1]), ([64, 200], [130, 257]), ([1, 33, 0, 129, 2], [300, 0, 40, 128, 77]),
    ([260, 90], [5, 700])], ids=["short", "two", "mixed", "tall"])
def test_many_rows(heads, kv, d, bs, nq, nk, dtype):
    CrossCase(12, nq, nk, num_heads=heads, kv_heads=kv, head_size=d, block_size=bs,
              dtype=dtype).check()


@BOTH
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nk", [([1], [9000]), ([100], [7000]), ([300], [5000]),
                                   ([1, 40], [6001, 3999])], ids=str)
def test_long_keys(nq, nk, d, dtype):
    # the keys of one row are split over many blocks of the grid and joined
    CrossCase(13, nq, nk, num_heads=2, kv_heads=1, head_size=d, block_size=16,
              dtype=dtype).check()


@BOTH
@pytest.mark.parametrize("nq", [[1, 1, 2], [150, 1, 40]], ids=str)
def test_unmapped_blocks(nq, dtype):
    CrossCase(14, nq, [300, 90, 500], num_heads=4, kv_heads=2, head_size=128, block_size=16,
              dtype=dtype, holes=5).check()
    CrossCase(15, nq, [30, 0, 5], num_heads=4, kv_heads=2, head_size=64, block_size=32,
              dtype=dtype, holes=1).check()    # the longest row sees nothing


@pytest.mark.parametrize("nq", [[1, 1, 1, 1], [40, 1, 70, 2]], ids=str)
def test_bad_sequences_and_uncovered_rows(nq):
    c = CrossCase(16, nq, [50, 60, 70, 80], num_heads=4, kv_heads=2, head_size=64,
                  block_size=16, pad=5)
    c.check()                                        # rows behind the last sequence: zero
    c.check(nk=[50, -1, 70, 80])                     # a negative length
    c.check(nk=[50, 60, 70, 2000])                   # past the table
    T = c.q.shape[0]
    c.check(cu=np.array([0, nq[0], nq[0] + nq[1], T + 1, T + 3]))
    c.check(cu=np.array([2, nq[0] + 1, nq[0] + nq[1], T - 5, T - 5]))   # rows 0 and 1 uncovered


def test_max_query_len():
    c = CrossCase(17, [1, 2, 1, 40], [50, 60, 70, 80], num_heads=4, kv_heads=2, head_size=64,
                  block_size=16)
    c.check(max_query_len=40)
    c.check(max_query_len=39)      # the last sequence is refused
    c.check(max_query_len=1)
    c.check(max_query_len=1 << 30)


@BOTH
@pytest.mark.parametrize("nq", [[1, 2], [70, 5]], ids=str)
def test_steep_and_flat_scores(nq, dtype):
    kw = dict(num_heads=4, kv_heads=1, head_size=128, block_size=16, dtype=dtype)
    CrossCase(18, nq, [400, 333], spread=3.0, **kw).check()     # one state takes it all
    CrossCase(19, nq, [400, 333], scale=-0.2, **kw).check()     # a negative scale
    CrossCase(20, nq, [400, 333], scale=1e-6, **kw).check()


def _values(c, out, rows):
    return out.float().reshape(-1, c.hq, c.d)[rows]


@BOTH
@pytest.mark.parametrize("nq", [[1, 1], [50, 20]], ids=str)
def test_infinities(nq, dtype):
    # states whose score is -inf weigh nothing; a row of nothing else is empty; a state of
    # score +inf has no finite softmax
    c = CrossCase(21, nq, [40, 200], num_heads=2, kv_heads=1, head_size=64, block_size=8,
                  dtype=dtype)
    c.q = c.q.abs() + 0.1
    first = [int(x) for x in c.table[0, :5]]
    c.k[first] = 0.0
    c.k[first, :, :, 0] = float("-inf")
    at = int(c.table[1, 3])
    c.k[at, 2] = c.k[at, 2] * 0
    c.k[at, 2, :, 5] = float("-inf")
    out, lse, status = c.gpu()
    assert status == 0
    assert (_values(c, out, slice(0, nq[0])) == 0).all()
    assert torch.isneginf(lse[:nq[0]]).all()
    rest = _values(c, out, slice(nq[0], None))
    assert torch.isfinite(rest).all() and torch.isfinite(lse[nq[0]:]).all()
    c.nk = [40, 200]
    ref = c.oracle()
    live = slice(nq[0], None)
    assert np.allclose(rest.numpy(), ref[0][live], atol=3e-2)
    c.k[at, 2, :, 5] = float("inf")
    out, lse, _ = c.gpu()
    assert not torch.isfinite(lse[nq[0]:]).any()


def test_equal_calls_give_equal_bits_and_fresh_workspace():
    c = CrossCase(22, [1, 130, 3, 1], [3000, 900, 40, 777], num_heads=8, kv_heads=2,
                  head_size=128, block_size=16)
    a = c.gpu()
    n = B.pkv_cross_attention_workspace_size(B.make_cross_args(
        c.q, c.k, c.v, torch.zeros(5), torch.zeros(4), torch.zeros(c.table.shape), c.q,
        num_heads=8, kv_num_heads=2))
    ws = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device=DEV)   # NaN everywhere
    b = c.gpu(workspace=ws[:n] if ws.data_ptr() % 256 == 0 else None)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert (ws[n:] == 0xFF).all()
    assert torch.equal(c.gpu(lse=False)[0], a[0])


def test_side_stream_and_graph_of_two_calls():
    c = CrossCase(23, [1, 60, 1], [500, 300, 9], num_heads=4, kv_heads=2, head_size=64,
                  block_size=16, dtype="bf16")
    want = c.gpu()
    dev = [x.to(DEV) for x in (c.q, c.k, c.v)] + [i32(x) for x in (c.cu, c.nk, c.table)]
    kw = dict(num_heads=4, kv_num_heads=2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    on_side = B.pkv_cross_attention(*dev, stream=side, **kw)
    torch.cuda.synchronize()
    assert torch.equal(on_side.cpu(), want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        one = B.pkv_cross_attention(*dev, **kw)
        two = B.pkv_cross_attention(one, *dev[1:], **kw)   # queries made by the first call
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(one.cpu(), want[0])
    c.q = want[0]
    assert torch.equal(two.cpu(), c.gpu()[0])


def test_two_streams_at_once():
    a = CrossCase(24, [1] * 30, [400] * 30, num_heads=8, kv_heads=2, head_size=128, block_size=16)
    b = CrossCase(25, [90] * 6, [900] * 6, num_heads=8, kv_heads=2, head_size=128, block_size=16)
    want = a.gpu()[0], b.gpu()[0]
    dev = [[x.to(DEV) for x in (c.q, c.k, c.v)] + [i32(x) for x in (c.cu, c.nk, c.table)]
           for c in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for d, s in zip(dev, streams):
            with torch.cuda.stream(s):
                got.append(B.pkv_cross_attention(*d, num_heads=8, kv_num_heads=2))
    torch.cuda.synchronize()
    for i, x in enumerate(got):
        assert torch.equal(x.cpu(), want[i % 2])


def test_more_rows_than_one_scan():
    # more sequences than a block's prefix table has entries
    rng = np.random.default_rng(3)
    n = 3000
    nq = [int(x) for x in rng.integers(0, 3, n)]
    nk = [int(x) for x in rng.integers(0, 40, n)]
    nq[1500], nk[1500] = 70, 300
    CrossCase(26, nq, nk, num_heads=2, kv_heads=1, head_size=64, block_size=16).check()


def test_merges_with_the_scores_of_another_cache():
    # two halves of a sequence's states, joined by their lse, give the whole
    c = CrossCase(27, [1, 40], [512, 256], num_heads=4, kv_heads=2, head_size=128, block_size=16)
    whole, lse = c.check()
    parts = []
    for half in (0, 1):
        table = np.full_like(c.table, -1)
        nk = [256, 128]
        for b, n in enumerate(nk):
            table[b, :n // 16] = c.table[b, half * n // 16:(half + 1) * n // 16]
        parts.append(c.check(table=table, nk=nk))
    w = [torch.exp(p[1].double() - lse.double())[..., None] for p in parts]
    both = sum(x * p[0].double().reshape(-1, 4, 128) for x, p in zip(w, parts))
    assert torch.allclose(both, whole.double().reshape(-1, 4, 128), atol=4 * 2.0 ** -11)


@pytest.mark.parametrize("nq", [[1, 2], [140, 33]], ids=str)
def test_cache_past_32_bit_offsets(nq):
    # the same states at blocks behind 2^31 elements and 2^32 bytes of each cache
    c = CrossCase(32, nq, [300, 77], num_heads=8, kv_heads=8, head_size=128, block_size=16)
    want = c.gpu()
    blocks = c.k.shape[0]
    first = 2 ** 31 // (16 * 8 * 128) + 5
    k = torch.empty((first + blocks, 16, 8, 128), dtype=c.t, device=DEV)
    v = torch.empty_like(k)
    k[first:], v[first:] = c.k.to(DEV), c.v.to(DEV)
    out = B.pkv_cross_attention(c.q.to(DEV), k, v, i32(c.cu), i32(c.nk),
                                i32(np.where(c.table >= 0, c.table + first, -1)),
                                num_heads=8, kv_num_heads=8)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want[0])


@pytest.mark.parametrize("heads,kv", [(3, 3), (5, 5), (6, 6), (12, 12), (7, 1), (11, 1), (9, 3),
                                      (24, 24), (20, 4)])
def test_head_counts(heads, kv):
    # kv heads that neighbouring warps take together: 8, 4, 2 or 1; rows that do not fill a tile
    for nq in ([1, 1, 2], [50, 3, 200]):
        CrossCase(33, nq, [130, 0, 700], num_heads=heads, kv_heads=kv, head_size=64,
                  block_size=16).check()


@pytest.mark.parametrize("d", [64, 128])
def test_many_whole_tiles(d):
    # more tiles than twice the SMs: dealt out whole, the rest cut; sequences of one tile, of many,
    # and empty ones between them
    rng = np.random.default_rng(4)
    nq = [int(x) for x in rng.integers(0, 90, 60)] + [700, 1, 0, 2]
    nk = [int(x) for x in rng.integers(0, 400, 60)] + [150, 900, 30, 0]
    CrossCase(34, nq, nk, num_heads=16, kv_heads=8, head_size=d, block_size=16).check()


def test_many_whole_tiles_of_more_sequences_than_one_scan():
    rng = np.random.default_rng(5)
    nq = [int(x) for x in rng.integers(0, 40, 1500)]
    nk = [int(x) for x in rng.integers(0, 60, 1500)]
    CrossCase(35, nq, nk, num_heads=2, kv_heads=1, head_size=64, block_size=16).check()


def test_few_tiles_cut_in_step():
    # ranges cut into pieces of their own (several kv heads, few tiles), uneven lengths
    for nk in ([5000, 0, 3000], [130, 9000, 400], [128 * 31, 128 * 33, 1]):
        CrossCase(36, [100, 30, 129], nk, num_heads=8, kv_heads=4, head_size=64, block_size=64,
                  dtype="bf16").check()


@pytest.mark.parametrize("d,bs", [(128, 128), (128, 32), (64, 128)])
def test_few_rows_of_tiles_under_load(d, bs):
    # one half of rows, both halves at work on it, tiles arriving in any order: equal bits each time
    c = CrossCase(37, [5] * 64, [4000] * 64, num_heads=8, kv_heads=2, head_size=d, block_size=bs)
    first, _ = c.check()
    for _ in range(10):
        assert torch.equal(c.gpu()[0], first)


@pytest.mark.parametrize("d", [64, 128])
def test_tiles_of_one_step_and_of_many(d):
    # tiles that one half works on alone, then tiles of both: equal bits each time
    rng = np.random.default_rng(6)
    nk = [int(x) for x in rng.choice([1, 90, 128, 129, 300, 1500], 200)]
    nq = [int(x) for x in rng.choice([20, 33, 70], 200)]
    c = CrossCase(38, nq, nk, num_heads=4, kv_heads=2, head_size=d, block_size=32)
    first, _ = c.check()
    for _ in range(10):
        assert torch.equal(c.gpu()[0], first)


@pytest.mark.parametrize("d,bs,nk", [(64, 16, 500), (128, 8, 120), (64, 24, 2000), (128, 16, 700)])
@pytest.mark.parametrize("batch,kv,heads", [(1, 1, 1), (3, 5, 15), (37, 2, 8), (70, 4, 4)])
def test_few_and_short_sequences(batch, kv, heads, d, bs, nk):
    # one launch for these, an even share of many steps for others: lengths of 0, 1 and all between,
    # several rows a sequence, rows that no sequence covers
    rng = np.random.default_rng(batch + d)
    keys = [int(x) for x in rng.integers(0, nk + 1, batch)]
    keys[0], keys[-1] = nk, min(1, nk)
    nq = [int(x) for x in rng.integers(0, 4, batch)]
    nq[0] = 3
    c = CrossCase(39, nq, keys, num_heads=heads, kv_heads=kv, head_size=d, block_size=bs, pad=300)
    c.check(max_query_len=3)


def _pieces(seed, dtype="f16"):
    # ranges that are cut, so that the workspace is used; and few and many rows in one call
    return CrossCase(seed, [1, 70, 2, 1], [9000, 4000, 70, 12000], num_heads=8, kv_heads=2,
                     head_size=128, block_size=16, dtype=dtype)


class _Call:
    def __init__(self, c):
        self.k = dict(num_heads=c.hq, kv_num_heads=c.hkv)
        self.a = [c.q.to(DEV), c.k.to(DEV), c.v.to(DEV), i32(c.cu), i32(c.nk), i32(c.table)]

    def __call__(self, **kw):
        return B.pkv_cross_attention(*self.a, **self.k, **kw)


def test_own_workspaces_of_threads_and_streams():
    calls = [_Call(_pieces(40)), _Call(_pieces(41))]
    size = 64 << 20
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    want = [c(workspace=ws) for c in calls]
    torch.cuda.synchronize()
    bad = []

    def work(c, expected, stream):
        with torch.cuda.stream(stream):
            got = [c() for _ in range(40)]
        torch.cuda.synchronize()
        bad.extend(i for i, g in enumerate(got) if not torch.equal(g, expected))

    one = torch.cuda.Stream()
    for streams in ((one, one), (one, torch.cuda.Stream())):   # two threads on one stream too
        threads = [threading.Thread(target=work, args=(c, w, s))
                   for c, w, s in zip(calls, want, streams)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not bad


def test_captured_call_beside_eager_ones():
    a, b = _Call(_pieces(42)), _Call(_pieces(43))
    want_a, want_b = a(), b()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = [a() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(side):
            graph.replay()
        eager = [b() for _ in range(6)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, want_a) for x in out)
        assert all(torch.equal(x, want_b) for x in eager)
