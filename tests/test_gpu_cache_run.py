"""The operators around the paged cache together, as a decoder with normed heads uses them: tables
from lengths, prompts normed, rotated and written, attended behind a sliding window in one
layer and behind what they share in another, samples forked from them, a step of single tokens,
beams that change places. Every step is checked against a 64-bit run of dense keys and values."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as orc
from paged_kv_cache_231_gb300 import binding as B

from .step_util import DEV, half_step, i32, wide

pytestmark = pytest.mark.gpu
HQ, HKV, D, BS, MB, NB = 8, 2, 64, 8, 24, 120
WINDOW, SINKS = 20, 3


class Decoder:
    """Two layers' pools; per row the 64-bit keys and values of both, rounded as the pools hold
    them."""

    def __init__(self, rows, dtype):
        self.gen = torch.Generator()
        self.gen.manual_seed(3)
        self.t, self.rows = dtype, rows
        self.pools = [self.new(NB, BS, HKV, D).to(DEV) for _ in range(4)]   # K V, K V
        self.table = torch.full((rows, MB), -1, dtype=torch.int32, device=DEV)
        self.past = i32([0] * rows)
        self.seen = [[] for _ in range(rows)]       # (k, v) of each layer, a token each
        ang = np.arange(300)[:, None] * 10000.0 ** (-np.arange(D // 2) / (D // 2))
        self.cos, self.sin = (torch.from_numpy(f(ang)).float().to(DEV) for f in (np.cos, np.sin))
        self.weights = [(1 + 0.2 * self.new(D)).to(self.t).to(DEV) for _ in range(2)]

    def new(self, *shape):
        return torch.randn(shape, generator=self.gen).to(self.t)

    def step(self, lengths, groups, shared, pad=0):
        T, n = sum(lengths) + pad, sum(lengths)
        cu, slots, pos, total, _ = B.pkv_paged_schedule(
            self.past, i32(lengths), self.table, num_blocks=NB, block_size=BS, num_tokens=T)
        outs = []
        for layer in (0, 1):
            q, k, v = self.new(T, HQ * D), self.new(T, HKV * D), self.new(T, HKV * D)
            kc, vc = self.pools[2 * layer:2 * layer + 2]
            rot = B.pkv_paged_append_norm_rotary(
                q.to(DEV), k.to(DEV), v.to(DEV), kc, vc, slots, pos.view(1, -1), num_heads=HQ,
                kv_num_heads=HKV, query_weight=self.weights[0], key_weight=self.weights[1],
                cos_cache=self.cos, sin_cache=self.sin, rotary_dim=D)
            same = dict(num_heads=HQ, kv_num_heads=HKV, max_query_len=max(lengths))
            if layer == 0:
                out = B.pkv_paged_window_attention(rot, kc, vc, cu, self.past, self.table,
                                                   window=WINDOW, sinks=SINKS, **same)
            else:
                out = B.pkv_paged_prefix_attention(rot, kc, vc, cu, self.past, self.table,
                                                   i32(groups), i32(shared), **same)
            torch.cuda.synchronize()
            outs.append(out)
            self.check(layer, lengths, q, k, v, rot, out, n)
        self.past = total.clone()

    def check(self, layer, lengths, q, k, v, rot, out, n):
        at, past = 0, self.past.tolist()
        q3, k3, v3 = (wide(x).reshape(q.shape[0], -1, D) for x in (q, k, v))
        qw, kw = (wide(w) for w in self.weights)
        for b, new in enumerate(lengths):
            for i in range(at, at + new):
                t = past[b] + i - at
                c, s = wide(self.cos)[t], wide(self.sin)[t]
                turn = lambda x: np.concatenate(  # noqa: E731
                    [x[:, :32] * c - x[:, 32:] * s, x[:, 32:] * c + x[:, :32] * s], 1)
                key = turn(orc.normed(k3[i][None], kw, 1e-6)[0])
                as_held = lambda x: wide(torch.from_numpy(x).to(self.t))  # noqa: E731
                if len(self.seen[b]) == t:
                    self.seen[b].append({})
                self.seen[b][t][layer] = as_held(key), v3[i]
                query = as_held(turn(orc.normed(q3[i][None], qw, 1e-6)[0]))
                # a key or query may be rounded to the other neighbour where it lies between two
                assert np.abs(wide(rot)[i].reshape(HQ, D) - query).max() <= \
                    2 * half_step(self.t) * np.abs(query).max() * 1.01
                j = [x for x in range(t + 1) if layer == 1 or x > t - WINDOW or x < SINKS]
                keys = np.repeat(np.stack([self.seen[b][x][layer][0] for x in j]), HQ // HKV, 1)
                values = np.repeat(np.stack([self.seen[b][x][layer][1] for x in j]), HQ // HKV, 1)
                score = np.einsum("hd,nhd->hn", query, keys) / 8
                w = np.exp(score - score.max(1, keepdims=True))
                ref = np.einsum("hn,nhd->hd", w / w.sum(1, keepdims=True), values)
                # Normed heads have elements of 0.8 on average. If all 64 of a key and of a query
                # were rounded to the other neighbour, by a step each, a score would be off by
                # 64 * 2 * 2 half steps * 0.64 / 8, 21 half steps; the weights and with them the
                # output (of values about 1) by as much, and by their own roundings: below 32.
                err = np.abs(wide(out)[i].reshape(HQ, D) - ref).max()
                assert err <= 32 * half_step(self.t), (b, t, layer, err)
            at += new
        assert not wide(out)[n:].any()               # rows behind the last sequence

    def fork(self, parents):
        before = [p.clone() for p in self.pools]
        past, table, free = B.pkv_paged_fork(i32(parents), self.past, self.table, self.pools)
        torch.cuda.synchronize()
        want = orc.fork(parents, self.past.tolist(), self.table.cpu().numpy(),
                        [wide(x) for x in before], num_blocks=NB, block_size=BS)
        assert past.tolist() == want[0] and (table.cpu().numpy() == want[1]).all()
        assert free.item() == want[2]
        assert all(np.array_equal(wide(x), y) for x, y in zip(self.pools, want[3]))
        self.past, self.table = past, table
        self.seen = [[dict(x) for x in self.seen[p]] if p >= 0 else [] for p in parents]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("sharing", [0, 1])
def test_prompts_samples_and_beams(dtype, sharing):
    B.pkv_testing_prefix_sharing(sharing)
    try:
        d = Decoder(8, dtype)
        d.step([37, 0, 0, 0, 50, 0, 0, 0], [0, 4, 8], [0, 0], pad=3)
        d.fork([0, 0, 0, 0, 4, 4, 4, -1])            # four samples of one, three of the other
        for _ in range(3):
            d.step([1, 1, 1, 1, 1, 1, 1, 0], [0, 4, 8], [32, 48], pad=1)
        d.fork([1, 1, 0, -1, 6, 4, 4, 2])            # beams change places, one moves over
        d.step([1, 2, 1, 0, 9, 1, 1, 1], [0, 3, 4, 7], [32, 0, 48])
        d.step([1, 1, 1, 12, 1, 1, 1, 1], [0, 3, 4, 7, 8], [32, 0, 48, 5])
        d.fork([-1] * 7 + [7])
        d.step([5, 0, 0, 0, 0, 0, 0, 1], [0, 8], [0])
    finally:
        B.pkv_testing_prefix_sharing()
