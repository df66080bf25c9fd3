"""CPU definitions, in 64 bits, of the operators around the paged cache: append with norms,
causal attention with a window or behind a shared prefix, forks of the block table's rows.
Test infrastructure only; shares no code with the GPU path."""
from __future__ import annotations

import numpy as np

from .step_oracle import BAD_BLOCK, BAD_SEQUENCE, NO_BLOCKS, append_axes


def normed(x, weight, epsilon):
    """x [tokens, heads, D]; a weight of None: as it is."""
    if weight is None:
        return x.copy()
    mean = (x ** 2).mean(-1, keepdims=True)
    return x / np.sqrt(mean + epsilon) * weight


def append_norm(q, k, v, *args, query_weight, key_weight, epsilon, **kw):
    """As step_oracle.append_axes, with the norms in front."""
    q = None if q is None else normed(q, query_weight, epsilon)
    return append_axes(q, normed(k, key_weight, epsilon), v, *args, **kw)


def causal_attention(q, key_cache, value_cache, cu, past, table, *, num_heads, kv_num_heads,
                     scale, window=0, sinks=0, max_query_len=0):
    """fp64 arrays: q [T, Hq, D], caches [NB, BS, Hkv, D]. Returns (out, lse, size, reach,
    status), as step_oracle.cross_attention."""
    T, Hq, D = q.shape
    NB, BS = key_cache.shape[:2]
    G, MB = Hq // kv_num_heads, table.shape[1]
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    size, reach, status = np.zeros((T, Hq, D)), np.zeros((T, Hq)), 0
    for b in range(len(past)):
        lo, hi, p = int(cu[b]), int(cu[b + 1]), int(past[b])
        if (lo < 0 or hi < lo or hi > T or not 0 <= p <= MB * BS or
                (max_query_len and hi - lo > max_query_len)):
            status |= BAD_SEQUENCE
            continue
        for i in range(lo, hi):
            t = p + i - lo
            j = np.arange(t + 1)
            if window > 0:
                j = j[(j > t - window) | (j < sinks)]
            if len(j) and j[-1] >= MB * BS:
                status |= BAD_BLOCK
                j = j[j < MB * BS]
            blk = table[b, j // BS]
            live = (blk >= 0) & (blk < NB)
            if not live.all():
                status |= BAD_BLOCK
            j, blk = j[live], blk[live]
            if not len(j):
                continue
            k = key_cache[blk, j % BS]                            # [n, Hkv, D]
            v = value_cache[blk, j % BS]
            x = q[i].reshape(kv_num_heads, G, D)
            s = scale * np.einsum("hgd,nhd->hgn", x, k)
            m = s.max(-1, keepdims=True)
            w = np.exp(s - m)
            total = w.sum(-1, keepdims=True)
            w = w / total
            out[i] = np.einsum("hgn,nhd->hgd", w, v).reshape(Hq, D)
            size[i] = np.einsum("hgn,nhd->hgd", w, np.abs(v)).reshape(Hq, D)
            lse[i] = (m + np.log(total))[..., 0].reshape(Hq)
            reach[i] = (abs(scale) * np.einsum("hgd,nhd->hgn", np.abs(x), np.abs(k))
                        ).max(-1).reshape(Hq)
    return out, lse, size, reach, status


def prefix_status(groups, shared, batch):
    """What is wrong with the groups of a prefix attention."""
    g = [int(x) for x in groups]
    bad = any(x < 0 or x > batch for x in g) or any(a > b for a, b in zip(g, g[1:]))
    return BAD_SEQUENCE if bad or any(int(s) < 0 for s in shared) else 0


def fork(parents, past, table, caches, *, num_blocks, block_size):
    """Rows one after the other. caches: arrays [num_blocks, block_size, ...]. Returns (new
    past, new table, free blocks, new caches, status)."""
    table = np.array(table, np.int64)
    B, MB = table.shape
    status, rows = 0, []
    for p in map(int, parents):
        n = 0
        if p >= B:
            status |= BAD_SEQUENCE
        elif p >= 0:
            n = int(past[p])
            if n < 0:
                status, n = status | BAD_SEQUENCE, 0
            elif n > MB * block_size:
                status, n = status | BAD_BLOCK, 0
        rows.append((p, n))
    new = np.full_like(table, -1)
    asks = []
    for b, (p, n) in enumerate(rows):
        if n == 0:
            continue
        held, rest = -(-n // block_size), n % block_size
        new[b, :held] = table[p, :held]
        first = rows[p][0] != p and not any(rows[x][0] == p for x in range(b))
        last = table[p, held - 1]
        if rest and p != b and not first and 0 <= last < num_blocks:
            new[b, held - 1] = -1
            asks.append((b, int(last), rest))
    taken = set()
    for b, (p, n) in enumerate(rows):
        for x in table[p, :-(-n // block_size)] if n else ():
            if x != -1 and not 0 <= x < num_blocks:
                status |= BAD_BLOCK
        taken |= {int(x) for x in new[b] if 0 <= x < num_blocks}
    free = [x for x in range(num_blocks) if x not in taken]
    caches = [c.copy() for c in caches]
    lengths, used = [n for _, n in rows], 0
    for b, last, rest in asks:
        if used == len(free):
            status, new[b], lengths[b] = status | NO_BLOCKS, -1, 0
            continue
        new[b, lengths[b] // block_size] = free[used]
        for c in caches:
            c[free[used], :rest] = c[last, :rest]
        used += 1
    return lengths, new, len(free) - used, caches, status
