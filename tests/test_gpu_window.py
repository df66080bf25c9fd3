"""GPU parity of pkv_paged_window_attention."""
import numpy as np
import pytest
import torch

from paged_kv_cache_231_gb300 import binding as B

from .cache_util import CausalCase
from .step_util import DEV, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 5), (1, 0), (1, 1), (7, 0), (16, 4), (33, 2),
                                          (64, 40), (100, 64), (100, 130), (1000, 3), (5, 500),
                                          (1 << 40, 1 << 40)])
@pytest.mark.parametrize("head_size,dtype", [(64, "f16"), (128, "bf16")])
def test_single_tokens(window, sinks, head_size, dtype):
    CausalCase(1, [1] * 9, [0, 1, 5, 15, 16, 17, 100, 200, 500], window=window, sinks=sinks,
               head_size=head_size, dtype=dtype, block_size=16).check()


@pytest.mark.parametrize("heads,kv", [(1, 1), (2, 2), (6, 2), (8, 2), (16, 2), (16, 1), (32, 2),
                                      (5, 1), (14, 2)])
@pytest.mark.parametrize("nq", [1, 2, 4, 5])
def test_tokens_and_heads(heads, kv, nq):
    CausalCase(2, [nq] * 5, [0, 3, 40, 129, 300], num_heads=heads, kv_heads=kv, window=50,
               sinks=3, block_size=8).check(max_query_len=nq)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (63, 1), (64, 0), (65, 4), (127, 0),
                                          (128, 16), (129, 130), (300, 4), (1000, 0)])
@pytest.mark.parametrize("head_size,dtype,heads,kv", [(64, "bf16", 4, 4), (128, "f16", 8, 2),
                                                      (128, "bf16", 6, 2), (64, "f16", 16, 1)])
def test_prompts(window, sinks, head_size, dtype, heads, kv):
    CausalCase(3, [1, 2, 17, 64, 0, 100, 300], [0, 3, 128, 500, 9, 0, 257], window=window,
               sinks=sinks, head_size=head_size, dtype=dtype, num_heads=heads, kv_heads=kv,
               block_size=32).check()


@pytest.mark.parametrize("block_size", [1, 3, 8, 16, 24, 40, 64, 100, 128, 256])
@pytest.mark.parametrize("window", [0, 77])
def test_block_sizes(block_size, window):
    CausalCase(4, [1, 150, 4, 40], [70, 333, 12, 0], window=window, sinks=5, head_size=128,
               num_heads=4, kv_heads=2, block_size=block_size).check()


@pytest.mark.parametrize("heads", [1, 3, 5, 7, 9, 11, 13, 15])
def test_odd_groups_in_tiles(heads):
    CausalCase(5, [200, 90, 33], [0, 401, 60], window=130, sinks=9, num_heads=heads, kv_heads=1,
               head_size=64, block_size=16).check()


@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 4), (1000, 140)])
@pytest.mark.parametrize("head_size", [64, 128])
def test_long_prompts(window, sinks, head_size):
    CausalCase(6, [700, 1, 513], [900, 2100, 0], window=window, sinks=sinks, num_heads=2,
               kv_heads=1, head_size=head_size, dtype="bf16", block_size=64).check()


@pytest.mark.parametrize("free", [False, True])
def test_unseen_blocks_may_be_gone(free):
    c = CausalCase(7, [1, 1, 60, 130], [300, 90, 400, 700], window=40, sinks=4, block_size=8,
                   free_unseen=free)
    c.check(status=0)


def test_holes_that_are_seen():
    c = CausalCase(8, [1, 3, 60, 1], [100, 90, 200, 50], window=64, sinks=4, block_size=8,
                   holes=((0, 0), (0, 9), (2, 20), (3, 6)))
    c.check(status=B.DEV_BAD_BLOCK)
    # the row's own key as well: nothing is left for it
    c = CausalCase(9, [1, 1], [8, 8], window=1, block_size=8, holes=((0, 1),))
    out, lse = c.check(status=B.DEV_BAD_BLOCK)
    assert not out[0].any() and torch.isneginf(lse[0]).all()


def test_holes_that_nobody_sees():
    CausalCase(10, [1, 60], [200, 200], window=64, sinks=4, block_size=8,
               holes=((0, 1), (0, 5), (1, 2), (1, 15))).check(status=0)


def test_keys_past_the_table():
    for nq in (1, 40):
        c = CausalCase(11, [nq, nq], [100, 20], block_size=8, window=30)
        c.table = np.ascontiguousarray(c.table[:, :13])      # 104 keys
        c.check(status=B.DEV_BAD_BLOCK if 100 + nq > 104 else 0)


@pytest.mark.parametrize("nq", [2, 70])
def test_bad_sequences(nq):
    c = CausalCase(12, [nq] * 4, [20, 30, 0, 50], window=25, sinks=1, pad=3)
    c.past[1] = -1
    out, lse = c.check(status=B.DEV_BAD_SEQUENCE)
    assert not out[nq:2 * nq].any() and torch.isneginf(lse[4 * nq:]).all()
    c.past[1] = 30
    c.cu = np.array([0, nq, 2 * nq, nq, 4 * nq], np.int32)
    ref = c.oracle()
    out, lse, status = c.gpu()
    assert status == ref[4]      # the last one has rows of two others, and too many keys
    assert np.allclose(out[:nq].double().numpy(), ref[0][:nq].reshape(nq, -1), atol=2e-2)
    c.cu = np.array([0, nq, 2 * nq, 3 * nq, 4 * nq], np.int32)
    c.check(max_query_len=nq)
    out, lse, status = c.gpu(max_query_len=nq - 1)
    assert status == B.DEV_BAD_SEQUENCE and not out.any()
    for past in (2 ** 31 - 1, c.table.shape[1] * c.bs + 1):
        c.past[2] = past
        c.check(status=B.DEV_BAD_SEQUENCE)


@pytest.mark.parametrize("spread,scale", [(4.0, 0.0), (1.0, 0.5), (1.0, -0.25), (0.0, 0.0)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_scores(spread, scale, dtype):
    CausalCase(13, [1, 90, 3], [300, 120, 0], window=100, sinks=8, spread=spread, scale=scale,
               dtype=dtype, head_size=128).check()


def test_many_sequences():
    rng = np.random.default_rng(14)
    nq = rng.choice([0, 1, 1, 1, 2, 9, 40], 1500)
    past = rng.integers(0, 90, 1500)
    CausalCase(14, nq, past, num_heads=2, kv_heads=1, window=33, sinks=2, block_size=8).check()


def test_without_lse_and_equal_bits():
    c = CausalCase(15, [1, 300, 2], [900, 40, 30], window=200, sinks=4, head_size=128)
    a, _, _ = c.gpu(lse=False)
    b, _, _ = c.gpu()
    assert torch.equal(a, b)


def test_no_tokens():
    c = CausalCase(16, [0, 0], [3, 0])
    out, lse, status = c.gpu()
    assert out.shape[0] == 0 and status == 0


def test_captured_and_replayed():
    c = CausalCase(17, [1, 200, 3], [800, 10, 90], window=150, sinks=4, head_size=128)
    want, wlse, _ = c.gpu()
    a = c.device()
    out = torch.zeros_like(a[0])
    lse = torch.zeros((a[0].shape[0], c.hq), device=DEV)
    kw = dict(num_heads=c.hq, kv_num_heads=c.hkv, window=c.window, sinks=c.sinks, output=out,
              lse=lse)
    B.pkv_paged_window_attention(*a, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.pkv_paged_window_attention(*a, **kw)
    for _ in range(3):
        out.zero_()
        lse.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want) and torch.equal(lse.cpu(), wlse)
    a[4].copy_(i32([300, 0, 7]))      # other lengths in the same graph
    c.past = [300, 0, 7]
    g.replay()
    torch.cuda.synchronize()
    again, _, _ = c.gpu()             # one row sees cache rows of NaN now: compared bit by bit
    assert torch.equal(out.cpu().view(torch.int16), again.view(torch.int16))


def test_other_stream():
    c = CausalCase(18, [1, 200, 3], [800, 10, 90], window=150, sinks=4)
    want, _, _ = c.gpu()
    a = c.device()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = B.pkv_paged_window_attention(*a, num_heads=c.hq, kv_num_heads=c.hkv, window=c.window,
                                       sinks=c.sinks, stream=s)
    s.synchronize()
    assert torch.equal(out.cpu(), want)


def _by_torch(c, lengths):
    """64 bits on the GPU: each row over the keys of its window and the sinks (one kv head)."""
    dev = c.device()
    past, cu, table = c.past, c.cu, dev[5].long()
    out, lse = [], []
    for b, n in enumerate(lengths):
        pos = past[b] + torch.arange(n, device=DEV)[:, None]
        j = torch.cat([pos - torch.arange(c.window, device=DEV),
                       torch.arange(c.sinks, device=DEV).expand(n, -1)], 1)
        seen = j >= 0
        seen[:, c.window:] &= j[:, c.window:] <= pos - c.window
        at = j.clamp(min=0)
        row = table[b, at // c.bs] * c.bs + at % c.bs
        k, v = (x.reshape(-1, c.d)[row].double() for x in dev[1:3])
        q = dev[0][cu[b]:cu[b + 1]].view(n, c.hq, c.d).double()
        s = torch.einsum("thd,tnd->thn", q, k) * c.d ** -0.5
        s = s.masked_fill(~seen[:, None], float("-inf"))
        lse.append(torch.logsumexp(s, -1))
        p = torch.softmax(s, -1)
        v = torch.where(seen[..., None], v, torch.zeros_like(v))
        out.append(torch.einsum("thn,tnd->thd", p, v))
    return torch.cat(out), torch.cat(lse)


@pytest.mark.parametrize("lengths", [[70000], [30000, 1, 0, 50000, 3], [66] * 1300], ids=len)
def test_more_tiles_than_a_plan_lists(lengths):
    # 16 heads to a kv head: tiles of 16 positions, up to 5000 of them
    c = CausalCase(19, lengths, [9] * len(lengths), num_heads=16, kv_heads=1, window=48, sinks=5,
                   block_size=16)
    out, lse, status = c.gpu()
    assert status == 0
    ref, rlse = _by_torch(c, lengths)
    # values of about 1: weights and output are rounded by half a step each; scores of a few units
    # err by 2^-17 of their magnitudes' sum, below 2^-11
    assert (out.to(DEV).view(ref.shape).double() - ref).abs().max() <= 8 * 2.0 ** -11
    assert (lse.to(DEV).double() - rlse).abs().max() <= 2.0 ** -10
