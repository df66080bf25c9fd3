"""Inputs and error bounds shared by the tests of the step operators."""
import numpy as np
import torch

from oracle import step_oracle as orc
from paged_kv_cache_231_gb300 import binding as B

DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"f16": B.PKV_F16, "bf16": B.PKV_BF16, "f32": B.PKV_F32}


def half_step(t):
    """Largest relative error of one rounding to t."""
    return torch.finfo(t).eps / 2


def wide(t):
    return t.detach().cpu().double().numpy()


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


def paged_pool(rng, lengths, block_size, max_blocks=None, spare=3):
    """A block table of shuffled blocks for rows of these lengths. Returns (table, blocks)."""
    need = [-(-n // block_size) for n in lengths]
    blocks = sum(need) + spare
    mb = max(need + [1]) if max_blocks is None else max_blocks
    ids = rng.permutation(blocks)
    table, at = np.full((len(lengths), mb), -1, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, blocks


def cross_bound(t, ref, lse, size, reach, n, values):
    """Bounds on |out - ref| and |lse - ref| of the cross attention.

    Scores: products of the inputs are exact in fp32; a sum of D <= 128 of them errs by at
    most D * 2^-24 = 2^-17 of the sum of magnitudes, which scaled is `reach`, whatever its
    order; the scaling and the log2 units cost a few half steps more, within that:
    ds = 2^-17 * reach. exp2 is good to 2^-21.
    A weight then errs by 2 ds + 2^-21 relative to the sum's other weights, plus one
    rounding to t for the product with v (half_step); in fp16 a weight below 2^-14 errs by
    2^-25 absolute against a largest weight of at least 1. Sums of n terms: n * 2^-23.
    The result is rounded once."""
    ds = 2.0 ** -17 * reach
    rel = 2 * ds + 2.0 ** -21 + half_step(t) + (n + 64) * 2.0 ** -23
    tiny = 2.0 ** -25 * n * values if t == torch.float16 else 0.0
    out = size * rel[..., None] * 1.01 + tiny + half_step(t) * np.abs(ref) * 1.01 + 1e-7
    live = np.where(np.isfinite(lse), lse, 0.0)
    return out, 2 * ds + (n + 64) * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * np.abs(live)


class CrossCase:
    """Ragged queries over paged encoder states, drawn from a seed; the cache rows that no
    state uses hold NaN."""

    def __init__(self, seed, nq, nk, *, num_heads, kv_heads, head_size, block_size,
                 dtype="f16", scale=0.0, spread=1.0, pad=0, max_blocks=None, holes=0):
        rng = np.random.default_rng(seed)
        gen = torch.Generator()
        gen.manual_seed(seed)
        self.t = TYPES[dtype]
        self.nq, self.nk, self.hq, self.hkv = nq, nk, num_heads, kv_heads
        self.d, self.bs = head_size, block_size
        self.table, blocks = paged_pool(rng, nk, block_size, max_blocks)
        self.cu = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
        T = int(self.cu[-1]) + pad
        new = lambda *shape: torch.randn(shape, generator=gen).mul(spread).to(self.t)  # noqa: E731
        self.q = new(T, num_heads * head_size)
        self.k = new(blocks, block_size, kv_heads, head_size)
        self.v = new(blocks, block_size, kv_heads, head_size)
        used = np.zeros((blocks, block_size), bool)
        for b, n in enumerate(nk):
            j = np.arange(n)
            used[self.table[b, j // block_size], j % block_size] = True
        unused = torch.from_numpy(~used)
        self.k[unused], self.v[unused] = float("nan"), float("nan")
        if holes:   # some blocks of the longest row are not there
            b = int(np.argmax(nk))
            n = -(-nk[b] // block_size)
            for c in rng.choice(n, min(holes, n), replace=False):
                self.table[b, c] = rng.choice([-1, blocks, blocks + 7, -5])
        self.scale = scale

    def gpu(self, *, max_query_len=0, lse=True, out=None, table=None, cu=None, nk=None, **kw):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = torch.full((self.q.shape[0], self.hq), float("nan"), device=DEV) if lse else None
        out = torch.full_like(self.q, float("nan"), device=DEV) if out is None else out
        B.pkv_cross_attention(
            self.q.to(DEV), self.k.to(DEV), self.v.to(DEV),
            i32(self.cu if cu is None else cu), i32(self.nk if nk is None else nk),
            i32(self.table if table is None else table), num_heads=self.hq,
            kv_num_heads=self.hkv, max_query_len=max_query_len, scale=self.scale,
            output=out, lse=got, device_status=status, **kw)
        torch.cuda.synchronize()
        return out.cpu(), None if got is None else got.cpu(), int(status.item())

    def oracle(self, *, max_query_len=0, table=None, cu=None, nk=None):
        shape = (-1, self.hq, self.d)
        return orc.cross_attention(
            wide(self.q).reshape(shape), wide(self.k), wide(self.v),
            self.cu if cu is None else cu, self.nk if nk is None else nk,
            self.table if table is None else table, num_heads=self.hq, kv_num_heads=self.hkv,
            scale=self.scale or self.d ** -0.5, max_query_len=max_query_len)

    def check(self, **kw):
        which = {k: v for k, v in kw.items() if k in ("max_query_len", "table", "cu", "nk")}
        out, lse, status = self.gpu(**kw)
        ref, rlse, size, reach, rstatus = self.oracle(**which)
        assert status == rstatus
        finite = self.v[~torch.isnan(self.v)].abs()
        values = float(finite.double().mean()) if finite.numel() else 0.0
        n = max(list(self.nk) + [1])
        tol, tol_lse = cross_bound(self.t, ref, rlse, size, reach, n, values)
        err = np.abs(wide(out).reshape(ref.shape) - ref)
        bad = ~(err <= tol)
        assert not bad.any(), (int(bad.sum()), float(np.nanmax(err)),
                               np.argwhere(bad)[:4].tolist())
        if lse is not None:
            empty = np.isneginf(rlse)
            assert (np.isneginf(lse.numpy()) == empty).all()
            dl = np.abs(wide(lse)[~empty] - rlse[~empty])
            assert (dl <= tol_lse[~empty]).all(), float(dl.max())
        return out, lse
