"""Step operators without a GPU: refusals of the C entries and of the binding, helper
functions, and the oracle against results worked out by hand."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import step_oracle as orc
from paged_kv_cache_231_gb300 import binding as B


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        from paged_kv_cache_231_gb300 import build
        build.build()
    return B.load_library()


P = 256   # a pointer that no refused call reads


def schedule_args(**kw):
    a = B.ScheduleArgs(P, P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 7 * P, None, 2, 8, 32, 16, 64)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(batch=0), 2), (dict(max_blocks=0), 2), (dict(num_blocks=0), 2),
    (dict(block_size=0), 2), (dict(num_tokens=-1), 2), (dict(batch=8193), 9),
    (dict(num_blocks=(1 << 20) + 1), 9), (dict(block_size=1 << 40), 9),
    (dict(max_blocks=1 << 40), 9), (dict(num_tokens=2**31 - 1), 9),
    (dict(max_blocks=1 << 27), 9),                      # max_blocks * block_size = 2^31
    (dict(max_blocks=2**31 - 10, block_size=1, batch=1), 9),
    (dict(num_blocks=1 << 20, block_size=1 << 11), 9),  # slots past 2^31
    (dict(past_seqlens=None), 1), (dict(new_seqlens=None), 1), (dict(block_table=None), 1),
    (dict(cumulative_sequence_length=None), 1), (dict(total_seqlens=P), 2),
])
def test_schedule_refusals(lib, change, status):
    before = B.pkv_launch_count()
    assert lib.pkv_paged_schedule(ctypes.byref(schedule_args(**change)), None) == status
    assert B.pkv_launch_count() == before


def axes_args(**kw):
    a = B.AppendAxesArgs(P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 7 * P, 8 * P, 9 * P, 10 * P,
                         None, 3, 4, 2, 64, 16, 8, 64, 100, 3, 0, B.PKV_F16, B.PKV_F32)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _axis(i, v):
    x = (ctypes.c_uint8 * 128)()
    x[i] = v
    return x


@pytest.mark.parametrize("change,status", [
    (dict(dtype=B.PKV_F32), 4), (dict(dtype=0), 4), (dict(table_dtype=B.PKV_BF16), 4),
    (dict(num_heads=3), 3), (dict(kv_num_heads=0), 3), (dict(num_tokens=-1), 2),
    (dict(head_size=0), 2), (dict(block_size=0), 2), (dict(num_blocks=0), 2),
    (dict(rotary_dim=63), 2), (dict(rotary_dim=66), 2), (dict(rotary_dim=-2), 2),
    (dict(num_axes=0), 2), (dict(num_axes=9), 2), (dict(rotary_positions=0), 2),
    (dict(pair_axis=_axis(31, 3)), 2), (dict(head_size=68), 9), (dict(head_size=264), 9),
    (dict(num_tokens=1 << 31), 9), (dict(key=None), 5), (dict(value=None), 5),
    (dict(query=None), 1), (dict(key_cache=None), 1), (dict(value_cache=None), 1),
    (dict(slot_mapping=None), 1), (dict(positions=None), 1), (dict(cos_cache=None), 1),
    (dict(sin_cache=None), 1), (dict(query=P + 8), 8), (dict(key=P + 2), 8),
    (dict(value_cache=P + 4), 8), (dict(query_out=P + 8), 8), (dict(cos_cache=P + 2), 8),
    (dict(query_out=P), 2), (dict(key=None, value=None, query=None, query_out=None), 1),
])
def test_append_axes_refusals(lib, change, status):
    before = B.pkv_launch_count()
    a = axes_args(**change)
    assert lib.pkv_paged_append_rotary_axes(ctypes.byref(a), None) == status
    assert B.pkv_launch_count() == before


def test_append_axes_pair_axis_past_rotary_dim_is_not_read(lib):
    # an axis behind the last pair does not matter; nothing to do for no tokens
    a = axes_args(pair_axis=_axis(32, 200), num_tokens=0)
    assert lib.pkv_paged_append_rotary_axes(ctypes.byref(a), None) == 0


def cross_args(**kw):
    a = B.CrossAttentionArgs(P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 7 * P, 8 * P, None, 3, 2, 4,
                             2, 64, 16, 8, 6, 0, B.PKV_F16, 0.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(dtype=B.PKV_F32), 4), (dict(num_heads=3), 3), (dict(num_heads=0), 3),
    (dict(head_size=0), 2), (dict(block_size=0), 2), (dict(num_blocks=0), 2),
    (dict(batch=0), 2), (dict(max_blocks=0), 2), (dict(num_tokens=-1), 2),
    (dict(max_query_len=-1), 2), (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2),
    (dict(head_size=96), 9), (dict(num_heads=34), 9), (dict(max_blocks=1 << 28), 9),
    (dict(num_tokens=1 << 31), 9), (dict(query=None), 1), (dict(key_cache=None), 1),
    (dict(value_cache=None), 1), (dict(cumulative_sequence_length=None), 1),
    (dict(key_seqlens=None), 1), (dict(block_table=None), 1), (dict(output=None), 1),
    (dict(query=P + 8), 8), (dict(key_cache=P + 8), 8), (dict(output=P + 2), 8),
    (dict(lse=P + 2), 8),
])
def test_cross_refusals(lib, change, status):
    before = B.pkv_launch_count()
    n = ctypes.c_size_t(0)
    a = cross_args(**change)
    assert lib.pkv_cross_attention_workspace_size(ctypes.byref(a), ctypes.byref(n)) == status
    assert lib.pkv_cross_attention(ctypes.byref(a), P, 1 << 40, None) == status
    assert B.pkv_launch_count() == before


def test_cross_workspace_refusals(lib):
    a, n = cross_args(), ctypes.c_size_t(0)
    assert lib.pkv_cross_attention_workspace_size(ctypes.byref(a), ctypes.byref(n)) == 0
    assert n.value == 0      # few and short sequences need none
    a = cross_args(max_blocks=4096)
    assert lib.pkv_cross_attention_workspace_size(ctypes.byref(a), ctypes.byref(n)) == 0
    assert n.value > 0
    before = B.pkv_launch_count()
    for ws, size in ((None, n.value), (P, n.value - 1), (P + 128, n.value)):
        assert lib.pkv_cross_attention(ctypes.byref(a), ws, size, None) == 7
    assert lib.pkv_cross_attention(ctypes.byref(cross_args(num_tokens=0)), None, 0, None) == 0
    assert B.pkv_launch_count() == before
    # the output in the place of the query: tiles read rows that others have written
    assert lib.pkv_cross_attention(ctypes.byref(cross_args(output=P)), P, n.value, None) == 2
    assert B.pkv_launch_count() == before
    assert lib.pkv_cross_attention(None, P, n.value, None) == 1
    assert lib.pkv_paged_schedule(None, None) == 1
    assert lib.pkv_paged_append_rotary_axes(None, None) == 1


def test_binding_refusals():
    z = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype)  # noqa: E731
    f16 = torch.float16
    sched = dict(num_blocks=8, block_size=4, num_tokens=5)
    with pytest.raises(TypeError):
        B.pkv_paged_schedule(z(2).long(), z(2), z(2, 3), **sched)
    with pytest.raises(ValueError):   # one length short
        B.pkv_paged_schedule(z(2), z(1), z(2, 3), **sched)
    with pytest.raises(ValueError):
        B.pkv_paged_schedule(z(2), z(2), z(2, 3), slot_mapping=z(4), **sched)
    with pytest.raises(ValueError):   # columns of a wider table
        B.pkv_paged_schedule(z(2), z(2), z(2, 6)[:, :3], **sched)
    with pytest.raises(ValueError):   # not on a GPU
        B.pkv_paged_schedule(z(2), z(2), z(2, 3), **sched)
    pool, half = z(4, 8, 2, 64, dtype=f16), z(9, 32, dtype=f16)
    rows = dict(num_heads=4, kv_num_heads=2, cos_cache=half, sin_cache=half, rotary_dim=64)
    q, k = z(3, 256, dtype=f16), z(3, 128, dtype=f16)
    for kw, err in ((dict(slot_mapping=z(4)), ValueError), (dict(positions=z(3, 2)), ValueError),
                    (dict(positions=z(3)), ValueError), (dict(key=k.float()), TypeError),
                    (dict(key=z(3, 64, dtype=f16)), ValueError), (dict(positions=None), ValueError),
                    (dict(pair_axis=[0] * 31), ValueError), (dict(pair_axis=[0] * 31 + [300]), ValueError),
                    (dict(sin_cache=half[:8]), ValueError), (dict(sin_cache=half.float()), TypeError),
                    (dict(value_cache=pool[:3]), ValueError), (dict(key_cache=pool.float()), TypeError)):
        a = dict(query=q, key=k, value=k, key_cache=pool, value_cache=pool, slot_mapping=z(3),
                 positions=z(1, 3), **rows)
        a.update(kw)
        with pytest.raises(err):
            B.pkv_paged_append_rotary_axes(**a)
    for kw, err in ((dict(query=q.float()), TypeError), (dict(key_seqlens=z(3)), ValueError),
                    (dict(block_table=z(1, 4)), ValueError), (dict(lse=z(3, 4)), TypeError),
                    (dict(lse=z(3, 2, dtype=torch.float32)), ValueError),
                    (dict(value_cache=pool.bfloat16()), TypeError), (dict(num_heads=8), ValueError),
                    (dict(output=z(2, 256, dtype=f16)), ValueError), (dict(block_table=None), ValueError),
                    (dict(query=z(3, 512, dtype=f16)[:, :256]), ValueError), (dict(), ValueError)):
        a = dict(query=q, key_cache=pool, value_cache=pool, cumulative_sequence_length=z(3),
                 key_seqlens=z(2), block_table=z(2, 4), num_heads=4, kv_num_heads=2)
        a.update(kw)
        with pytest.raises(err):
            B.pkv_cross_attention(**a)


def test_rotary_pair_axis():
    assert B.rotary_pair_axis([2, 3, 1]) == [0, 0, 1, 1, 1, 2]
    assert B.rotary_pair_axis([3, 2, 1], by_turns=True) == [0, 1, 2, 0, 1, 0]
    assert B.rotary_pair_axis([0, 2]) == [1, 1]
    with pytest.raises(ValueError):
        B.rotary_pair_axis([])
    with pytest.raises(ValueError):
        B.rotary_pair_axis([2, -1])


def test_oracle_schedule_by_hand():
    # blocks of 4, pool of 8: row 0 holds 5 and 2 (7 tokens), row 1 idles with 1, row 2 is new
    table = np.array([[5, 2, -1], [1, -1, -1], [-1, -1, -1]])
    cu, slots, pos, total, free, new, st = orc.schedule(
        [7, 3, 0], [2, 0, 5], table, num_blocks=8, block_size=4, num_tokens=8)
    assert cu.tolist() == [0, 2, 2, 7] and total.tolist() == [9, 3, 5] and free == 2 and st == 0
    assert new.tolist() == [[5, 2, 0], [1, -1, -1], [3, 4, -1]]   # free: 0 3 4 6 7
    assert slots.tolist() == [11, 0, 12, 13, 14, 15, 16, -1]
    assert pos.tolist() == [7, 8, 0, 1, 2, 3, 4, -1]
    # a pool of 3: row 0 asks for the last one, row 2 gets nothing, a row without need does
    cu, slots, pos, total, free, new, st = orc.schedule(
        [4, 1, 0, 2], [1, 3, 1, 2], [[1, -1], [0, -1], [-1, -1], [0, -1]], num_blocks=3,
        block_size=4, num_tokens=9)
    assert cu.tolist() == [0, 1, 4, 4, 6] and total.tolist() == [5, 4, 0, 4]
    assert free == 0 and st == orc.NO_BLOCKS and slots.tolist()[:6] == [8, 1, 2, 3, 2, 3]


def test_oracle_append_by_hand():
    # one head of 4, pairs (0, 2) and (1, 3), a quarter turn on axis 1 for the second pair
    cos, sin = np.array([[1.0, 1.0], [0.0, 0.0]]), np.array([[0.0, 0.0], [1.0, 1.0]])
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    pool = np.zeros((2, 1, 4))
    qo, kc, vc, _, _, st = orc.append_axes(
        x, x, 2 * x, pool, pool, np.array([1]), np.array([[0], [1]]), cos, sin, num_heads=1,
        kv_num_heads=1, rotary_dim=4, pair_axis=[0, 1], interleaved=False, q_out=np.zeros((1, 1, 4)))
    assert qo[0, 0].tolist() == [1, -4, 3, 2] and kc[1, 0].tolist() == [1, -4, 3, 2]
    assert vc[1, 0].tolist() == [2, 4, 6, 8] and not kc[0].any() and st == 0


def test_oracle_cross_by_hand():
    k = np.zeros((2, 2, 1, 2))
    v = np.arange(8.0).reshape(2, 2, 1, 2)
    k[1, 0, 0] = [np.log(3.0), 0]     # the second state of the row below weighs 3
    q = np.array([[[1.0, 5.0]], [[0.0, 0.0]]])
    out, lse, _, _, st = orc.cross_attention(q, k, v, [0, 1, 2], [3, 0], np.array([[0, 1], [0, 1]]),
                                             num_heads=1, kv_num_heads=1, scale=1.0)
    assert np.allclose(out[0, 0], (v[0, 0, 0] + v[0, 1, 0] + 3 * v[1, 0, 0]) / 5)
    assert np.allclose(lse[0, 0], np.log(5.0))
    assert not out[1].any() and np.isneginf(lse[1, 0]) and st == 0
