"""GPU parity of pkv_paged_prefix_attention: the causal attention of every row over its own
table row, whatever is said to be shared."""
import numpy as np
import pytest
import torch

from paged_kv_cache_231_gb300 import binding as B

from .cache_util import CausalCase
from .step_util import DEV, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["whatever can be", "by the rule"], autouse=True)
def sharing(request):
    """Small cases would hardly share anything by the rule."""
    B.pkv_testing_prefix_sharing(1 if request.param == "whatever can be" else 0)
    yield request.param
    B.pkv_testing_prefix_sharing()


def case(seed, nq, own, groups, **kw):
    """own: tokens of each sequence behind what its group shares."""
    past, at = [], 0
    for n, keys in groups:
        past += [keys + own[at + i] for i in range(n)]
        at += n
    past += own[at:]
    return CausalCase(seed, nq, past, groups=groups, **kw)


@pytest.mark.parametrize("head_size,dtype,heads,kv", [(64, "f16", 4, 2), (128, "bf16", 8, 2),
                                                      (64, "bf16", 3, 1), (128, "f16", 4, 4)])
@pytest.mark.parametrize("shared", [16, 64, 144, 640])
def test_single_tokens(head_size, dtype, heads, kv, shared):
    case(1, [1] * 7, [0, 1, 5, 40, 17, 130, 9], [(7, shared)], head_size=head_size, dtype=dtype,
         num_heads=heads, kv_heads=kv).check(prefix=True, max_query_len=1)


@pytest.mark.parametrize("width", [1, 2, 3, 40, 100])
@pytest.mark.parametrize("heads", [1, 4])
def test_widths(width, heads):
    rng = np.random.default_rng(2)
    case(2, [1] * width, [int(x) for x in rng.integers(0, 50, width)], [(width, 160)],
         num_heads=heads, kv_heads=1).check(prefix=True)


@pytest.mark.parametrize("head_size,dtype,heads,kv", [(64, "f16", 4, 2), (128, "bf16", 8, 2),
                                                      (64, "bf16", 3, 1), (128, "f16", 4, 4)])
@pytest.mark.parametrize("block_size", [8, 24, 32])
def test_prompts_and_groups(head_size, dtype, heads, kv, block_size):
    n = block_size
    case(3, [30, 1, 0, 90, 64, 2, 7, 1, 200], [0, 3, 10, 50, 0, 200, 9, 100, 64],
         [(3, 10 * n), (1, 4 * n), (0, 5 * n), (4, 20 * n)], head_size=head_size, dtype=dtype,
         num_heads=heads, kv_heads=kv, block_size=block_size).check(prefix=True)


def test_what_is_shared_is_cut():
    # more than a sequence's past, than its table; nothing; groups that leave sequences out
    c = case(4, [1, 4, 1, 30, 1], [0, 7, 50, 2, 1], [(3, 64), (2, 320)])
    ref = c.oracle()
    for shared in ([64, 320], [32, 16], [0, 0], [1, 17], [63, 319], [48, 0]):
        c.check(prefix=True, shared=shared, reference=ref)
    c.check(prefix=True, groups=[1, 3], shared=[64], reference=ref)
    c.check(prefix=True, groups=[3, 5], shared=[256], reference=ref)
    c.check(prefix=True, groups=[0], shared=[], reference=ref)
    # a sequence of the group has a shorter past than the others share (its past ends with the
    # last block that all three have: with 33 the key behind it would not be shared)
    c = CausalCase(5, [1, 5, 1], [100, 32, 200], groups=[(3, 32)])
    c.check(prefix=True, shared=[400])
    c = CausalCase(6, [2, 2], [0, 0], groups=[(2, 0)])
    c.check(prefix=True, shared=[50])


def test_bad_groups():
    c = case(7, [1, 4, 1, 30, 1], [0, 7, 50, 2, 1], [(3, 64), (2, 320)])
    ref = c.oracle()
    for groups, shared in (([0, 3, 6], [64, 320]), ([-1, 3, 5], [64, 320]), ([0, 3, 2], [64, 320]),
                           ([3, 0, 5], [64, 64])):
        c.check(prefix=True, groups=groups, shared=shared, status=B.DEV_BAD_SEQUENCE, reference=ref)
    c.check(prefix=True, shared=[-1, 320], status=B.DEV_BAD_SEQUENCE, reference=ref)


def test_bad_sequences():
    for past in (-1, -2 ** 31):
        c = case(8, [1, 4, 1, 30, 1], [0, 7, 50, 2, 1], [(3, 64), (2, 320)], pad=2)
        c.past[1] = past
        out, lse = c.check(prefix=True, status=B.DEV_BAD_SEQUENCE)
        assert not out[1:5].any() and torch.isneginf(lse[-2:]).all()
    c = case(9, [1, 4, 1, 30, 1], [0, 7, 50, 2, 1], [(3, 64), (2, 320)])
    c.check(prefix=True, max_query_len=29, status=B.DEV_BAD_SEQUENCE)


def test_holes():
    c = case(10, [1, 4, 1, 40], [0, 7, 50, 2], [(4, 160)], block_size=16)
    c.table[:, 3] = -1                       # shared by all
    c.table[2, 11] = 10 ** 6                 # one row's own
    c.check(prefix=True, status=B.DEV_BAD_BLOCK)
    c = CausalCase(11, [1, 1], [64, 64], groups=[(2, 64)], block_size=16)
    c.table[:, :4] = -1
    c.table[1, 4] = -1                       # nothing is left for the second row
    out, lse = c.check(prefix=True, status=B.DEV_BAD_BLOCK)
    assert not out[1].any() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("scale,spread", [(0.0, 4.0), (-0.5, 1.0), (1.0, 1.0)])
def test_scores(scale, spread):
    case(12, [1] * 20 + [50], list(range(20)) + [9], [(21, 256)], scale=scale, spread=spread,
         head_size=128, dtype="bf16").check(prefix=True)


def test_many_groups():
    rng = np.random.default_rng(13)
    groups = [(int(n), 16 * int(k)) for n, k in zip(rng.integers(0, 6, 400),
                                                   rng.integers(0, 6, 400))]
    rows = sum(n for n, _ in groups)
    case(13, [int(x) for x in rng.choice([0, 1, 1, 2, 20], rows)],
         [int(x) for x in rng.integers(0, 40, rows)], groups, num_heads=2,
         kv_heads=1).check(prefix=True)


def test_equal_bits_and_graph():
    c = case(14, [1] * 30 + [70], list(range(30)) + [200], [(31, 512)], head_size=128)
    want, wlse, _ = c.gpu(prefix=True)
    again, alse, _ = c.gpu(prefix=True)
    assert torch.equal(want, again) and torch.equal(wlse, alse)
    a = c.device() + [i32(c.groups), i32(c.shared)]
    out = torch.zeros_like(a[0])
    kw = dict(num_heads=c.hq, kv_num_heads=c.hkv, output=out)
    B.pkv_paged_prefix_attention(*a, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.pkv_paged_prefix_attention(*a, **kw)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want)
    s = torch.cuda.Stream()
    other = B.pkv_paged_prefix_attention(*a, num_heads=c.hq, kv_num_heads=c.hkv, stream=s)
    s.synchronize()
    assert torch.equal(other.cpu(), want)


@pytest.mark.parametrize("nq,own,keys,heads,kv,head_size,dtype", [
    ([1] * 64, list(range(64)), 2048, 32, 8, 128, "f16"),        # single tokens, short own keys
    ([1] * 40, [0] * 39 + [3000], 4096, 16, 16, 64, "bf16"),     # one of them with many
    ([4] * 40, [9] * 40, 2048, 32, 8, 128, "bf16"),              # drafts: 16 rows of a kv head
    ([9] * 30, [5] * 30, 4096, 16, 16, 64, "f16"),               # rows of a tile's quarter
    ([200, 150], [0, 7], 1024, 8, 2, 128, "bf16"),               # nothing to gain
])
def test_sizes_that_the_rule_is_about(nq, own, keys, heads, kv, head_size, dtype, sharing):
    c = case(15, nq, own, [(len(nq), keys)], num_heads=heads, kv_heads=kv, head_size=head_size,
             dtype=dtype, block_size=16)
    ref = c.oracle()
    c.check(prefix=True, max_query_len=max(nq), reference=ref)
    c.check(prefix=True, reference=ref)            # the longest sequence is not named


def test_shared_or_not_is_the_same_but_for_rounding():
    c = case(16, [1] * 20 + [30], [7] * 20 + [40], [(21, 512)], head_size=128, dtype="bf16")
    B.pkv_testing_prefix_sharing(2)
    alone = c.gpu(prefix=True)
    B.pkv_testing_prefix_sharing(1)
    shared = c.gpu(prefix=True)
    same = c.gpu()                                 # the window attention without a window
    assert torch.equal(alone[0], same[0]) and torch.equal(alone[1], same[1])
    assert not torch.equal(alone[0], shared[0])    # the hook does what it says
    assert torch.allclose(alone[1], shared[1], atol=1e-5)


def test_workspace_given_and_refused():
    c = case(17, [1] * 6, [3] * 6, [(6, 256)])
    a = c.device() + [i32(c.groups), i32(c.shared)]
    want = c.gpu(prefix=True)[0]
    out = torch.empty_like(a[0])
    kw = dict(num_heads=c.hq, kv_num_heads=c.hkv)
    need = B.pkv_paged_prefix_attention_workspace_size(B.make_prefix_args(*a, out, **kw))
    ws = torch.full((max(need, 1) + 512,), 255, dtype=torch.uint8, device=DEV)
    B.pkv_paged_prefix_attention(*a, output=out, workspace=ws, **kw)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want)
    assert (ws[need:] == 255).all()


@pytest.mark.parametrize("nq", [1, 3])
@pytest.mark.parametrize("head_size,dtype,heads,kv", [(128, "f16", 8, 2), (64, "bf16", 4, 4)])
def test_few_tokens_beside_the_shared_keys(nq, head_size, dtype, heads, kv, sharing):
    # groups, rows of none, empty and bad sequences, padding: each row is written by one of three
    # kernels; the same bits eagerly, replayed and from a workspace full of something else
    lengths, own = [nq] * 40, [int(x) for x in np.random.default_rng(18).integers(0, 90, 40)]
    lengths[3] = lengths[17] = lengths[30] = 0
    c = case(18, lengths, own, [(14, 512), (2, 0), (16, 1024)], head_size=head_size, dtype=dtype,
             num_heads=heads, kv_heads=kv, pad=3)
    c.check(prefix=True, max_query_len=nq)
    c.past[35] = -1
    c.check(prefix=True, max_query_len=nq, status=B.DEV_BAD_SEQUENCE)
    a = c.device() + [i32(c.groups), i32(c.shared)]
    kw = dict(num_heads=heads, kv_num_heads=kv, max_query_len=nq)
    out = torch.empty_like(a[0])
    need = B.pkv_paged_prefix_attention_workspace_size(B.make_prefix_args(*a, out, **kw))
    ws = torch.zeros(need + 256, dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.pkv_paged_prefix_attention(*a, output=out, workspace=ws, **kw)
    want = c.gpu(prefix=True, max_query_len=nq)[0]
    for fill in (0, 255, 0x7f):
        out.fill_(float("nan"))
        ws.fill_(fill)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want)
