"""The step operators together, as a decoder with image inputs uses them: tables and slots
from request lengths, K / V and Q with positions of several axes into the pool, causal paged
attention over it, encoder states in a second pool, cross attention over those."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as orc
from paged_kv_cache_231_gb300 import binding as B

from .step_util import DEV, half_step, i32, wide

pytestmark = pytest.mark.gpu
HQ, HKV, D, BS, AXES = 4, 2, 64, 8, 3


def test_three_steps_of_a_decoder():
    gen = torch.Generator()
    gen.manual_seed(5)
    new = lambda *s: torch.randn(s, generator=gen).half()  # noqa: E731
    rows, mb, nb = 4, 16, 40
    pool = [new(nb, BS, HKV, D).to(DEV) for _ in range(4)]       # self K, V; encoder K, V
    table = torch.full((rows, mb), -1, dtype=torch.int32, device=DEV)
    etable = torch.full((rows, mb), -1, dtype=torch.int32, device=DEV)
    states = [30, 0, 11, 64]
    ang = np.arange(200)[:, None] * 10000.0 ** (-np.arange(D // 2) / (D // 2))
    cos, sin = (torch.from_numpy(f(ang)).float().to(DEV) for f in (np.cos, np.sin))
    axis = B.rotary_pair_axis([12, 10, 10])

    # encoder states: scheduled and written once, without positions
    zero = i32([0] * rows)
    ecu, eslots, *_ = B.pkv_paged_schedule(zero, i32(states), etable, num_blocks=nb,
                                           block_size=BS, num_tokens=sum(states))
    ek, ev = new(sum(states), HKV * D), new(sum(states), HKV * D)
    assert B.pkv_paged_append_rotary_axes(None, ek.to(DEV), ev.to(DEV), pool[2], pool[3], eslots,
                                          None, num_heads=HQ, kv_num_heads=HKV) is None

    past, seen = i32([0] * rows), [[] for _ in range(rows)]      # per row: (k, v) fp64 rows
    for lengths in ([20, 33, 0, 5], [1, 1, 7, 1], [1, 1, 1, 1]):
        T = sum(lengths) + 3                                     # a padded batch
        cu, slots, pos, total, free = B.pkv_paged_schedule(
            past, i32(lengths), table, num_blocks=nb, block_size=BS, num_tokens=T)
        axes = torch.stack([pos, pos // 2, pos % 5]).contiguous()
        q, k, v = new(T, HQ * D), new(T, HKV * D), new(T, HKV * D)
        rot = B.pkv_paged_append_rotary_axes(
            q.to(DEV), k.to(DEV), v.to(DEV), pool[0], pool[1], slots, axes, num_heads=HQ,
            kv_num_heads=HKV, cos_cache=cos, sin_cache=sin, rotary_dim=D, pair_axis=axis)
        # the rows stand in the pool already: no slot for the attention to write
        out = B.pkv_paged_attention(rot, k.to(DEV), v.to(DEV), pool[0], pool[1], cu, past, table,
                                    torch.full_like(slots, -1), num_heads=HQ, kv_num_heads=HKV)
        cross = B.pkv_cross_attention(out, pool[2], pool[3], cu, i32(states), etable,
                                      num_heads=HQ, kv_num_heads=HKV, max_query_len=max(lengths))
        torch.cuda.synchronize()
        n = sum(lengths)
        assert cu.tolist() == [0] + list(np.cumsum(lengths))
        # 64-bit run of the same step
        rows3 = [wide(x).reshape(T, -1, D) for x in (q, k, v)]
        rq, rk, rv, *_ = orc.append_axes(
            *rows3, np.zeros((T, HKV, D)), np.zeros((T, HKV, D)),
            np.where(np.arange(T) < n, np.arange(T), -1), axes.cpu().numpy(), wide(cos), wide(sin),
            num_heads=HQ, kv_num_heads=HKV, rotary_dim=D, pair_axis=axis, interleaved=False,
            q_out=np.zeros((T, HQ, D)))
        at = 0
        ref = np.zeros((n, HQ, D))
        for b, m in enumerate(lengths):
            for t in range(m):
                seen[b].append((rk[at], rv[at]))
                ks, vs = (np.repeat(np.stack(x), HQ // HKV, 1) for x in zip(*seen[b]))
                s = np.einsum("hd,nhd->hn", rq[at], ks) * D ** -0.5
                w = np.exp(s - s.max(-1, keepdims=True))
                ref[at] = np.einsum("hn,nhd->hd", w / w.sum(-1, keepdims=True), vs)
                at += 1
        got = wide(out)[:n].reshape(n, HQ, D)
        # rounded queries and keys move a score by 2 half steps of sum |q k| (below 60 here,
        # scaled 7.5), weights and result by one half step each
        e = half_step(torch.float16)
        assert np.abs(got - ref).max() <= (4 * 7.5 + 2) * e * max(1.0, np.abs(rv).max())
        rc, *_ = orc.cross_attention(
            wide(out)[:n].reshape(n, HQ, D), wide(pool[2]), wide(pool[3]), cu.cpu().numpy(), states,
            etable.cpu().numpy(), num_heads=HQ, kv_num_heads=HKV, scale=D ** -0.5)
        assert np.abs(wide(cross)[:n].reshape(n, HQ, D) - rc).max() <= 4 * e * max(1.0, np.abs(rv).max())
        past = total
    # the first request is done: its blocks serve the next one
    held = int((-(-past // BS)).sum())
    assert free.tolist() == [nb - held]
    past = past.clone()
    gone = set(table[0, :int(-(-past[0] // BS))].tolist())
    past[0] = 0
    table[0] = -1
    cu, slots, pos, total, free2 = B.pkv_paged_schedule(
        past, i32([BS * len(gone), 0, 0, 0]), table, num_blocks=nb, block_size=BS,
        num_tokens=BS * len(gone))
    assert free2.tolist() == free.tolist()
    assert cu.tolist() == [0] + [BS * len(gone)] * 4
    kept = {int(x) for b in range(1, 4) for x in table[b, :int(-(-past[b] // BS))]}
    assert not kept & {int(s) // BS for s in slots.tolist()}
