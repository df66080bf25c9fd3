"""Inputs shared by the tests of the causal paged attention (window, shared prefix)."""
import numpy as np
import torch

from oracle import cache_oracle as orc
from paged_kv_cache_231_gb300 import binding as B

from .step_util import DEV, TYPES, cross_bound, i32, paged_pool, wide


class CausalCase:
    """Ragged queries behind the tokens of a paged cache, drawn from a seed; cache rows that no
    token of the call sees hold NaN. groups: [(sequences, shared keys)] of sequences one after the
    other that begin with the same blocks (whole blocks, so shared keys are cut to them)."""

    def __init__(self, seed, nq, past, *, num_heads=4, kv_heads=2, head_size=64, block_size=16,
                 dtype="f16", window=0, sinks=0, scale=0.0, spread=1.0, pad=0, groups=(),
                 max_blocks=None, holes=(), free_unseen=False):
        rng = np.random.default_rng(seed)
        gen = torch.Generator()
        gen.manual_seed(seed)
        self.t = TYPES[dtype]
        self.nq, self.past, self.hq, self.hkv = list(nq), list(past), num_heads, kv_heads
        self.d, self.bs, self.window, self.sinks, self.scale = (head_size, block_size, window,
                                                                sinks, scale)
        lengths = [n + p for n, p in zip(nq, past)]
        self.table, blocks = paged_pool(rng, lengths, block_size, max_blocks)
        at, self.groups, self.shared = 0, [0], []
        for n, keys in groups:
            lead = keys // block_size
            for b in range(at, at + n):
                self.table[b, :lead] = self.table[at, :lead]
            at += n
            self.groups.append(at)
            self.shared.append(keys)
        self.cu = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
        T = int(self.cu[-1]) + pad
        new = lambda *shape: torch.randn(shape, generator=gen).mul(spread).to(self.t)  # noqa: E731
        self.q = new(T, num_heads * head_size)
        self.k = new(blocks, block_size, kv_heads, head_size)
        self.v = new(blocks, block_size, kv_heads, head_size)
        used, self.seen = np.zeros((blocks, block_size), bool), []
        for b, (n, p) in enumerate(zip(nq, past)):
            j = np.arange(n + p)
            if window > 0:
                j = j[(j > p - window) | (j < sinks)]
            j = j if n else j[:0]
            self.seen.append(j)
            used[self.table[b, j // block_size], j % block_size] = True
            if free_unseen:
                gone = np.setdiff1d(np.arange(self.table.shape[1]), j // block_size)
                self.table[b, gone] = rng.choice([-1, blocks, -7], len(gone))
        unused = torch.from_numpy(~used)
        self.k[unused], self.v[unused] = float("nan"), float("nan")
        for b, c in holes:
            self.table[b, c] = rng.choice([-1, blocks, blocks + 7, -5])

    def device(self):
        return [x.to(DEV) for x in (self.q, self.k, self.v)] + [
            i32(x) for x in (self.cu, self.past, self.table)]

    def gpu(self, *, prefix=False, max_query_len=0, lse=True, groups=None, shared=None, **kw):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = torch.full((self.q.shape[0], self.hq), float("nan"), device=DEV) if lse else None
        out = torch.full_like(self.q, float("nan"), device=DEV)
        a = self.device()
        same = dict(num_heads=self.hq, kv_num_heads=self.hkv, max_query_len=max_query_len,
                    scale=self.scale, output=out, lse=got, device_status=status, **kw)
        if prefix:
            B.pkv_paged_prefix_attention(
                *a, i32(self.groups if groups is None else groups),
                i32(self.shared if shared is None else shared), **same)
        else:
            B.pkv_paged_window_attention(*a, window=self.window, sinks=self.sinks, **same)
        torch.cuda.synchronize()
        return out.cpu(), None if got is None else got.cpu(), int(status.item())

    def oracle(self, max_query_len=0):
        return orc.causal_attention(
            wide(self.q).reshape(-1, self.hq, self.d), wide(self.k), wide(self.v), self.cu,
            self.past, self.table, num_heads=self.hq, kv_num_heads=self.hkv,
            scale=self.scale or self.d ** -0.5, window=self.window, sinks=self.sinks,
            max_query_len=max_query_len)

    def check(self, *, prefix=False, max_query_len=0, status=None, reference=None, **kw):
        out, lse, got = self.gpu(prefix=prefix, max_query_len=max_query_len, **kw)
        ref, rlse, size, reach, want = reference or self.oracle(max_query_len)
        assert got == (want if status is None else status)
        finite = self.v[~torch.isnan(self.v)].abs()
        values = float(finite.double().mean()) if finite.numel() else 0.0
        n = max([len(j) for j in self.seen] + [1])
        # a shared prefix: both parts' sums are brought to one maximum and added in 32 bits, some
        # 2^-20 of the size more
        tol, tol_lse = cross_bound(self.t, ref, rlse, size * (1 + 2.0 ** -10 * prefix), reach, n,
                                   values)
        tol = tol + 2.0 ** -19 * size * prefix
        err = np.abs(wide(out).reshape(ref.shape) - ref)
        bad = ~(err <= tol)
        assert not bad.any(), (int(bad.sum()), float(np.nanmax(err)),
                               np.argwhere(bad)[:4].tolist())
        if lse is not None:
            empty = np.isneginf(rlse)
            assert (np.isneginf(lse.numpy()) == empty).all()
            dl = np.abs(wide(lse)[~empty] - rlse[~empty])
            assert (dl <= tol_lse[~empty] + 2.0 ** -20 * prefix).all(), float(dl.max())
        return out, lse
