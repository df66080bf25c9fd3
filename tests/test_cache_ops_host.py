"""The operators around the paged cache without a GPU: refusals of the C entries and of the
binding, where the binding's memory comes from, and the oracle against results worked out by
hand."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache_oracle as orc
from paged_kv_cache_231_gb300 import binding as B

from .test_step_host import _axis, axes_args, lib  # noqa: F401 - a fixture
from .test_stream_memory import Stream, Tensor, f16, fake, i32  # noqa: F401 - a fixture

P = 256   # a pointer that no refused call reads


def refused(call, args, status, *more):
    before = B.pkv_launch_count()
    assert call(ctypes.byref(args), *more) == status
    assert B.pkv_launch_count() == before


# ---------------------------------------------------------------------------------- norm
def norm_args(**kw):
    own = {k: kw.pop(k) for k in list(kw) if k in ("query_weight", "key_weight", "epsilon",
                                                   "weight_dtype")}
    a = B.AppendNormArgs(axes_args(**kw), 11 * P, 12 * P, 1e-6, B.PKV_F32)
    for k, v in own.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(epsilon=0.0), 2), (dict(epsilon=-1.0), 2), (dict(epsilon=float("nan")), 2),
    (dict(epsilon=float("inf")), 2), (dict(weight_dtype=B.PKV_BF16), 4), (dict(weight_dtype=0), 4),
    (dict(query_weight=None, key_weight=None), 1), (dict(query_weight=P + 2), 8),
    (dict(key_weight=P + 1), 8), (dict(dtype=B.PKV_F32), 4), (dict(num_heads=3), 3),
    (dict(num_tokens=-1), 2), (dict(rotary_dim=66), 2), (dict(head_size=264), 9),
    (dict(pair_axis=_axis(31, 3)), 2), (dict(key=None), 5), (dict(query=None), 1),
    (dict(slot_mapping=None), 1), (dict(positions=None), 1), (dict(cos_cache=P + 2), 8),
    (dict(query=P + 8), 8), (dict(query_out=P), 2),
])
def test_append_norm_refusals(lib, change, status):  # noqa: F811
    refused(lib.pkv_paged_append_norm_rotary, norm_args(**change), status, None)


def test_append_norm_of_nothing(lib):  # noqa: F811
    refused(lib.pkv_paged_append_norm_rotary, norm_args(num_tokens=0), 0, None)
    assert lib.pkv_paged_append_norm_rotary(None, None) == 1


# ------------------------------------------------------------------------ window, prefix
def window_args(**kw):
    a = B.WindowAttentionArgs(P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 7 * P, 8 * P, None, 3, 2, 4,
                              2, 64, 16, 8, 6, 0, 10, 2, B.PKV_F16, 0.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def prefix_args(**kw):
    a = B.PrefixAttentionArgs(P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 7 * P, 8 * P, 9 * P, 10 * P,
                              None, 3, 2, 1, 4, 2, 64, 16, 8, 6, 0, B.PKV_F16, 0.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


SAME = [
    (dict(dtype=B.PKV_F32), 4), (dict(num_heads=3), 3), (dict(num_heads=0), 3),
    (dict(head_size=0), 2), (dict(block_size=0), 2), (dict(num_blocks=0), 2),
    (dict(batch=0), 2), (dict(max_blocks=0), 2), (dict(num_tokens=-1), 2),
    (dict(max_query_len=-1), 2), (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2),
    (dict(head_size=96), 9), (dict(num_heads=34), 9), (dict(max_blocks=1 << 28), 9),
    (dict(num_tokens=1 << 31), 9), (dict(query=None), 1), (dict(key_cache=None), 1),
    (dict(value_cache=None), 1), (dict(cumulative_sequence_length=None), 1),
    (dict(past_seqlens=None), 1), (dict(block_table=None), 1), (dict(output=None), 1),
    (dict(query=P + 8), 8), (dict(key_cache=P + 8), 8), (dict(output=P + 2), 8),
    (dict(lse=P + 2), 8),
]


@pytest.mark.parametrize("change,status", SAME + [(dict(window=-1), 2), (dict(sinks=-1), 2)])
def test_window_refusals(lib, change, status):  # noqa: F811
    n = ctypes.c_size_t(0)
    a = window_args(**change)
    assert lib.pkv_paged_window_attention_workspace_size(ctypes.byref(a), ctypes.byref(n)) == status
    refused(lib.pkv_paged_window_attention, a, status, P, 1 << 40, None)


@pytest.mark.parametrize("change,status", SAME + [
    (dict(num_groups=-1), 2), (dict(num_groups=1 << 31), 9), (dict(group_offsets=None), 1),
    (dict(shared_seqlens=None), 1)])
def test_prefix_refusals(lib, change, status):  # noqa: F811
    n = ctypes.c_size_t(0)
    a = prefix_args(**change)
    assert lib.pkv_paged_prefix_attention_workspace_size(ctypes.byref(a), ctypes.byref(n)) == status
    refused(lib.pkv_paged_prefix_attention, a, status, P, 1 << 40, None)


def test_workspaces(lib):  # noqa: F811
    n = ctypes.c_size_t(0)
    size = lambda call, a: (call(ctypes.byref(a), ctypes.byref(n)), n.value)  # noqa: E731
    win, pre = (lib.pkv_paged_window_attention_workspace_size,
                lib.pkv_paged_prefix_attention_workspace_size)
    assert size(win, window_args()) == (0, 0)              # few and short sequences
    # a window bounds what a long table is planned for
    long = dict(max_blocks=1 << 16, num_blocks=1 << 16)
    assert size(win, window_args(**long)) == (0, 0)
    assert size(win, window_args(window=0, **long))[1] > 0
    assert size(pre, prefix_args()) == (0, 0)              # nothing that sharing could save
    big = dict(num_tokens=64, batch=64, num_heads=32, kv_num_heads=8, head_size=128, **long)
    assert size(pre, prefix_args(**big))[1] >= 64 * 32 * 129 * 4
    assert size(pre, prefix_args(num_groups=0, **big))[1] < 64 << 20
    need = size(pre, prefix_args(**big))[1]
    for ws, k in ((None, need), (P, need - 1), (P + 128, need)):
        refused(lib.pkv_paged_prefix_attention, prefix_args(**big), 7, ws, k, None)
    need = size(win, window_args(window=0, **long))[1]
    for ws, k in ((None, need), (P, need - 1), (P + 128, need)):
        refused(lib.pkv_paged_window_attention, window_args(window=0, **long), 7, ws, k, None)
    for call, a in ((lib.pkv_paged_window_attention, window_args), (lib.pkv_paged_prefix_attention,
                                                                  prefix_args)):
        refused(call, a(num_tokens=0), 0, None, 0, None)
        refused(call, a(output=P), 2, P, 1 << 40, None)
        assert call(None, P, 1 << 40, None) == 1
    assert win(ctypes.byref(window_args()), None) == 1
    assert pre(ctypes.byref(prefix_args()), None) == 1


def test_sharing_hook(lib):  # noqa: F811
    n = ctypes.c_size_t(0)
    a = prefix_args()
    try:
        B.pkv_testing_prefix_sharing(1)
        lib.pkv_paged_prefix_attention_workspace_size(ctypes.byref(a), ctypes.byref(n))
        assert n.value > 0
    finally:
        B.pkv_testing_prefix_sharing()
    for mode in (-1, 3):
        with pytest.raises(B.PagedKVError):
            B.pkv_testing_prefix_sharing(mode)


# ---------------------------------------------------------------------------------- fork
def fork_args(caches=(P, 2 * P), rows=(16, 32), **kw):
    n = len(caches)
    at, width = (ctypes.c_int64 * max(n, 1))(*caches), (ctypes.c_int64 * max(n, 2))(*rows)
    a = B.ForkArgs(P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, ctypes.addressof(at),
                   ctypes.addressof(width), None, 2, 8, 32, 16, n)
    a.keep = (at, width)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(batch=0), 2), (dict(max_blocks=0), 2), (dict(num_blocks=0), 2), (dict(block_size=0), 2),
    (dict(num_caches=-1), 2), (dict(batch=8193), 9), (dict(num_blocks=(1 << 20) + 1), 9),
    (dict(block_size=1 << 40), 9), (dict(max_blocks=1 << 40), 9), (dict(max_blocks=1 << 27), 9),
    (dict(num_blocks=1 << 20, block_size=1 << 11), 9), (dict(num_caches=257), 9),
    (dict(parents=None), 1), (dict(past_seqlens=None), 1), (dict(block_table=None), 1),
    (dict(new_past_seqlens=None), 1), (dict(new_block_table=None), 1), (dict(caches=()), 0),
    (dict(rows=(16, 0)), 2), (dict(rows=(16, -16)), 2), (dict(rows=(16, 24)), 9),
    (dict(rows=(1 << 31, 16)), 9), (dict(rows=(1 << 27, 16)), 9), (dict(caches=(P, 0)), 1),
    (dict(caches=(P, P + 8)), 8), (dict(new_past_seqlens=2 * P), 2),
    (dict(new_block_table=3 * P), 2), (dict(free_blocks=P), 2),
])
def test_fork_refusals(lib, change, status):  # noqa: F811
    a = fork_args(**change)
    n = ctypes.c_size_t(0)
    assert lib.pkv_paged_fork_workspace_size(ctypes.byref(a), ctypes.byref(n)) == status
    if status:
        refused(lib.pkv_paged_fork, a, status, P, 1 << 40, None)


def test_fork_workspace(lib):  # noqa: F811
    n = ctypes.c_size_t(0)
    a = fork_args()
    assert lib.pkv_paged_fork_workspace_size(ctypes.byref(a), ctypes.byref(n)) == 0
    assert n.value == 256 + 16 * 2      # what the binding makes
    for ws, k in ((None, n.value), (P, n.value - 1), (P + 128, n.value)):
        refused(lib.pkv_paged_fork, a, 7, ws, k, None)
    a.caches = None
    assert lib.pkv_paged_fork_workspace_size(ctypes.byref(a), ctypes.byref(n)) == 1
    assert lib.pkv_paged_fork(None, P, 1 << 40, None) == 1


# ------------------------------------------------------------------------------- binding
def test_binding_refusals():
    z = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype)  # noqa: E731
    half = torch.float16
    pool, table = z(4, 8, 2, 64, dtype=half), z(9, 32, dtype=half)
    q, k, w = z(3, 256, dtype=half), z(3, 128, dtype=half), z(64, dtype=half)
    rows = dict(num_heads=4, kv_num_heads=2, cos_cache=table, sin_cache=table, rotary_dim=64)
    for kw, err in ((dict(query_weight=None), ValueError), (dict(query_weight=w[:32]), ValueError),
                    (dict(query_weight=w.double()), TypeError), (dict(key_weight=w.float()), TypeError),
                    (dict(slot_mapping=None), ValueError), (dict(positions=z(3)), ValueError),
                    (dict(key=k.float()), TypeError), (dict(pair_axis=[0] * 31), ValueError),
                    (dict(key_cache=pool[0]), ValueError), (dict(), ValueError)):
        a = dict(query=q, key=k, value=k, key_cache=pool, value_cache=pool, slot_mapping=z(3),
                 positions=z(1, 3), query_weight=w, **rows)
        a.update(kw)
        with pytest.raises(err):
            B.pkv_paged_append_norm_rotary(**a)
    same = ((dict(query=q.float()), TypeError), (dict(past_seqlens=z(3)), ValueError),
            (dict(past_seqlens=z(2).long()), TypeError), (dict(block_table=z(1, 4)), ValueError),
            (dict(lse=z(3, 4)), TypeError), (dict(lse=z(3, 2, dtype=torch.float32)), ValueError),
            (dict(value_cache=pool.bfloat16()), TypeError), (dict(num_heads=8), ValueError),
            (dict(output=z(2, 256, dtype=half)), ValueError), (dict(block_table=None), ValueError),
            (dict(query=z(3, 512, dtype=half)[:, :256]), ValueError),
            (dict(key_cache=pool.transpose(1, 2)), ValueError), (dict(), ValueError))
    for kw, err in same:
        a = dict(query=q, key_cache=pool, value_cache=pool, cumulative_sequence_length=z(3),
                 past_seqlens=z(2), block_table=z(2, 4), num_heads=4, kv_num_heads=2)
        a.update(kw)
        with pytest.raises(err):
            B.pkv_paged_window_attention(window=5, **a)
        with pytest.raises(err):
            B.pkv_paged_prefix_attention(group_offsets=z(2), shared_seqlens=z(1), **a)
    for kw, err in ((dict(group_offsets=z(1)), ValueError), (dict(shared_seqlens=None), ValueError),
                    (dict(shared_seqlens=z(1).long()), TypeError)):
        a = dict(query=q, key_cache=pool, value_cache=pool, cumulative_sequence_length=z(3),
                 past_seqlens=z(2), block_table=z(2, 4), num_heads=4, kv_num_heads=2,
                 group_offsets=z(2), shared_seqlens=z(1))
        a.update(kw)
        with pytest.raises(err):
            B.pkv_paged_prefix_attention(**a)
    for kw, err in ((dict(parents=None), ValueError), (dict(parents=z(3)), ValueError),
                    (dict(past_seqlens=z(2).long()), TypeError),
                    (dict(new_block_table=z(2, 3)), ValueError), (dict(caches=[pool]), ValueError),
                    (dict(free_blocks=z(2)), ValueError), (dict(), ValueError)):
        a = dict(parents=z(2), past_seqlens=z(2), block_table=z(2, 4), num_blocks=8, block_size=4)
        a.update(kw)
        with pytest.raises(err):
            B.pkv_paged_fork(**a)


class Pool(Tensor):
    def element_size(self):
        return 2


def test_fork_looks_at_its_caches():
    one = Pool((4, 8, 2, 64), f16)
    narrow = Pool((4, 8, 16), f16)
    at, rows, blocks, size = B._cache_rows([one, one, narrow])
    assert rows == [256, 256, 32] and (blocks, size) == (4, 8) and at == [4096] * 3
    for bad in (Pool((5, 8, 16), f16), Pool((4, 16), f16), Pool((4,), f16)):
        with pytest.raises(ValueError):
            B._cache_rows([one, bad])
    strided = Pool((4, 8, 2, 64), f16)
    strided.is_contiguous = lambda: False
    with pytest.raises(ValueError):
        B._cache_rows([one, strided])
    elsewhere = Pool((4, 8, 2, 64), f16)
    elsewhere.get_device = lambda: 1
    with pytest.raises(ValueError):
        B._cache_rows([one, elsewhere])


def norm(**kw):
    rows = Tensor((3, 256), f16)
    return [B.pkv_paged_append_norm_rotary(rows, Tensor((3, 128), f16), Tensor((3, 128), f16),
                                           Tensor((4, 8, 2, 64), f16), Tensor((4, 8, 2, 64), f16),
                                           Tensor((3,), i32), None, num_heads=4, kv_num_heads=2,
                                           key_weight=Tensor((64,), f16), **kw)]


def causal(call, *more):
    pool = Tensor((4, 8, 2, 64), f16)

    def run(**kw):
        return [call(Tensor((3, 256), f16), pool, pool, Tensor((3,), i32), Tensor((2,), i32),
                     Tensor((2, 4), i32), *more, num_heads=4, kv_num_heads=2, **kw)]
    return run


window = causal(B.pkv_paged_window_attention)
prefix = causal(B.pkv_paged_prefix_attention, Tensor((2,), i32), Tensor((1,), i32))


def fork(**kw):
    return B.pkv_paged_fork(Tensor((2,), i32), Tensor((2,), i32), Tensor((2, 4), i32),
                            [Pool((4, 8, 2, 64), f16)] * 2, **kw)


CALLS = pytest.mark.parametrize("call", [norm, window, prefix, fork])


@pytest.fixture
def spaces(fake, monkeypatch):  # noqa: F811
    monkeypatch.setattr(B, "_window_workspace", lambda *a: 1 << 20)
    monkeypatch.setattr(B, "_prefix_workspace", lambda *a: 1 << 20)
    return fake


@CALLS
@pytest.mark.parametrize("capturing", [False, True])
def test_another_stream(spaces, call, capturing):
    side = Stream(7, capturing)
    returned = call(stream=side)
    assert spaces.made and all(t.made_on is side for t in spaces.made)
    for t in spaces.made:   # what the caller gets is used on the current stream too
        assert t.recorded == ([spaces.main] if any(t is r for r in returned) else [])
    assert spaces.calls[0][1][-1] == 7 and spaces.now is spaces.main


@CALLS
def test_the_current_stream(spaces, call):
    call()
    assert spaces.made and all(t.made_on is spaces.main and not t.recorded for t in spaces.made)
    assert spaces.calls[0][1][-1] == 1


@pytest.mark.parametrize("off", range(6))
@pytest.mark.parametrize("device", [-1, 1])
def test_each_tensor_has_to_be_on_the_current_device(spaces, off, device):
    a = [Tensor((3, 256), f16), Tensor((4, 8, 2, 64), f16), Tensor((4, 8, 2, 64), f16),
         Tensor((3,), i32), Tensor((2,), i32), Tensor((2, 4), i32)]
    a[off].get_device, a[off].is_cuda = lambda: device, device >= 0
    with pytest.raises(ValueError):
        B.pkv_paged_window_attention(*a, num_heads=4, kv_num_heads=2)
    assert not spaces.calls


@pytest.mark.parametrize("call", [window, fork])
def test_a_workspace_is_kept(spaces, call):
    call()
    n = [t for t in spaces.made if t.dtype is spaces.uint8]
    call()
    assert len(n) == 1 and [t for t in spaces.made if t.dtype is spaces.uint8] == n


def test_a_large_prefix_workspace_is_not_kept(spaces, monkeypatch):
    for need, kept in ((64 << 20, True), ((64 << 20) + 1, False)):
        B._OWN.__dict__.clear()
        monkeypatch.setattr(B, "_prefix_workspace", lambda *a: need)
        prefix()
        assert bool(B._OWN.__dict__) == kept


# -------------------------------------------------------------------------------- oracle
def test_oracle_norm_by_hand():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    assert np.allclose(orc.normed(x, np.array([1.0, 2.0, 3.0, 4.0]), 0.0), [[[1.2, 3.2, 0, 0]]])
    assert np.allclose(orc.normed(x, np.ones(4), 18.75), x / 5)
    assert (orc.normed(x, None, 1.0) == x).all()


def test_oracle_window_by_hand():
    # keys of zero weigh the same: the outputs are means of the values 0 .. 7 that a row sees
    k, v = np.zeros((4, 2, 1, 1)), np.arange(8.0).reshape(4, 2, 1, 1)
    q, table = np.zeros((3, 1, 1)), np.array([[0, 1, 2, 3]])
    run = lambda **kw: orc.causal_attention(q, k, v, [0, 3], [4], table, num_heads=1,  # noqa: E731
                                            kv_num_heads=1, scale=1.0, **kw)
    out, lse, _, _, st = run()
    assert out.ravel().tolist() == [2.0, 2.5, 3.0] and st == 0
    assert np.allclose(lse.ravel(), np.log([5, 6, 7]))
    assert run(window=2)[0].ravel().tolist() == [3.5, 4.5, 5.5]
    assert np.allclose(run(window=2, sinks=1)[0].ravel(), [7 / 3, 3.0, 11 / 3])
    assert np.allclose(run(window=4, sinks=3)[0].ravel(), [2.0, 2.5, 21 / 7])
    out, lse, _, _, st = orc.causal_attention(q, k, v, [0, 3], [4], table[:, :2], num_heads=1,
                                              kv_num_heads=1, scale=1.0, window=2)
    assert st == orc.BAD_BLOCK and out[0, 0, 0] == 3.0 and np.isneginf(lse[1:]).all()
    st = orc.causal_attention(q, k, v, [0, 3], [9], table, num_heads=1, kv_num_heads=1, scale=1.0)[-1]
    assert st == orc.BAD_SEQUENCE


def test_oracle_fork_by_hand():
    # blocks of 4; row 0 holds 2 5 and two tokens of 1, row 1 holds 3 whole
    table = [[2, 5, 1], [3, -1, -1], [-1, -1, -1], [-1, -1, -1]]
    cache = np.arange(8 * 4).reshape(8, 4)
    past, new, free, (c,), st = orc.fork([0, 1, 0, 1], [10, 4, 0, 0], table, [cache], num_blocks=8,
                                         block_size=4)
    assert past == [10, 4, 10, 4] and free == 3 and st == 0     # of 0 4 6 7
    assert new.tolist() == [[2, 5, 1], [3, -1, -1], [2, 5, 0], [3, -1, -1]]
    assert c[0].tolist() == [4, 5, 2, 3] and (c[1:] == cache[1:]).all()
    # row 0 goes over to row 2 alone: its block goes with it; row 1 ends
    past, new, free, (c,), st = orc.fork([-1, -1, 0, -1], [10, 4, 0, 0], table, [cache],
                                         num_blocks=8, block_size=4)
    assert past == [0, 0, 10, 0] and new[2].tolist() == [2, 5, 1] and free == 5
    assert (c == cache).all() and st == 0
    # a pool without a free block
    past, new, free, _, st = orc.fork([0, 0, 0, 1], [10, 4, 0, 0], table, [], num_blocks=6,
                                      block_size=4)
    assert past == [10, 10, 10, 4] and free == 0 and new[1].tolist() == [2, 5, 0]
    past, new, free, _, st = orc.fork([0, 0, 0, 0], [10, 4, 0, 0], table, [], num_blocks=6,
                                      block_size=4)
    assert past == [10, 10, 10, 10] and new[2:, 2].tolist() == [3, 4] and st == 0
