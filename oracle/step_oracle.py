"""CPU definitions, in 64 bits, of the step operators: schedule, append with rotary axes,
cross attention. Test infrastructure only; shares no code with the GPU path."""
from __future__ import annotations

import numpy as np

BAD_BLOCK, BAD_SLOT, BAD_POSITION, BAD_SEQUENCE, NO_BLOCKS = 1, 2, 4, 8, 64


def schedule(past, new, table, *, num_blocks, block_size, num_tokens):
    """Rows one after the other. Returns (cu, slots, positions, total, free, table, status)."""
    table = np.array(table, np.int64)
    B, MB = table.shape
    limit, status = MB * block_size, 0
    up = lambda x: -(-max(x, 0) // block_size)  # noqa: E731
    rows = []
    for p, n in zip(map(int, past), map(int, new)):
        if p < 0 or n < 0:
            status, n = status | BAD_SEQUENCE, 0
        if p > limit or n > limit - max(p, 0):
            status, n = status | BAD_BLOCK, 0
        rows.append((p, n, min(up(p), MB)))
    held = set()
    for b, (_, _, h) in enumerate(rows):
        for x in table[b, :h]:
            if 0 <= x < num_blocks:
                held.add(int(x))
            elif x != -1:
                status |= BAD_BLOCK
    free = [x for x in range(num_blocks) if x not in held]
    slots, positions = np.full(num_tokens, -1), np.full(num_tokens, -1)
    cu, total, asked, used = [0], [], 0, 0
    tokens = 0   # granted before the token buffers are looked at
    for b, (p, n, h) in enumerate(rows):
        need = up(p + n) - h if n else 0
        first, asked = asked, asked + need
        if need and asked > len(free):
            status, n = status | NO_BLOCKS, 0
        elif n:
            tokens += n
            if tokens > num_tokens:
                status, n = status | BAD_SEQUENCE, 0
        if n:
            table[b, h:h + need] = free[first:asked]
            used += need
            for t in range(n):
                blk = table[b, (p + t) // block_size]
                if not 0 <= blk < num_blocks:
                    status |= BAD_BLOCK
                else:
                    slots[cu[-1] + t] = blk * block_size + (p + t) % block_size
                positions[cu[-1] + t] = p + t
        total.append(p + n)
        cu.append(cu[-1] + n)
    return (np.array(cu), slots, positions, np.array(total), len(free) - used, table, status)


def append_axes(q, k, v, key_cache, value_cache, slots, positions, cos, sin, *, num_heads,
                kv_num_heads, rotary_dim, pair_axis, interleaved, q_out):
    """fp64 arrays; q [T, Hq, D] or None, k and v [T, Hkv, D], caches [rows, Hkv, D]. Returns
    (q_out, key_cache, value_cache, slack, status): slack as q_out and key_cache, the size of
    the products that meet in each element."""
    T, _, D = k.shape
    kc, vc = key_cache.copy(), value_cache.copy()
    qo = None if q_out is None else q_out.copy()
    slack_q = None if qo is None else np.zeros_like(qo)
    slack_k, status = np.zeros_like(kc), 0
    half = rotary_dim // 2

    def turned(x, t):
        out, size = x.copy(), np.zeros_like(x)
        for j in range(half):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            row = positions[pair_axis[j], t]
            c, s = cos[row, j], sin[row, j]
            out[:, a] = x[:, a] * c - x[:, b] * s
            out[:, b] = x[:, b] * c + x[:, a] * s
            size[:, a] = abs(x[:, a] * c) + abs(x[:, b] * s)
            size[:, b] = abs(x[:, b] * c) + abs(x[:, a] * s)
        return out, size

    for t in range(T):
        if slots[t] < 0:
            continue
        known = all(0 <= positions[pair_axis[j], t] < len(cos) for j in range(half))
        fits = slots[t] < kc.shape[0]
        status |= (0 if known else BAD_POSITION) | (0 if fits else BAD_SLOT)
        if qo is not None:
            qo[t], slack_q[t] = turned(q[t], t) if known else (q[t], 0.0)
        if known and fits:
            kc[slots[t]], slack_k[slots[t]] = turned(k[t], t)
            vc[slots[t]] = v[t]
    return qo, kc, vc, slack_q, slack_k, status


def cross_attention(q, key_cache, value_cache, cu, klen, table, *, num_heads, kv_num_heads,
                    scale, max_query_len=0):
    """fp64 arrays: q [T, Hq, D], caches [NB, BS, Hkv, D]. Returns (out, lse, size, reach,
    status): size [T, Hq, D] = sum_j w_j |v_j| / sum_j w_j, reach [T, Hq] = the largest
    scale * sum_d |q_d k_jd| of a row (both for error bounds)."""
    T, Hq, D = q.shape
    NB, BS = key_cache.shape[:2]
    G, MB = Hq // kv_num_heads, table.shape[1]
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    size, reach, status = np.zeros((T, Hq, D)), np.zeros((T, Hq)), 0
    for b in range(len(klen)):
        lo, hi, n = int(cu[b]), int(cu[b + 1]), int(klen[b])
        if lo < 0 or hi < lo or hi > T or n < 0 or (max_query_len and hi - lo > max_query_len):
            status |= BAD_SEQUENCE
            continue
        if hi == lo:
            continue
        if n > MB * BS:
            status, n = status | BAD_BLOCK, MB * BS
        j = np.arange(n)
        blk = table[b, j // BS]
        live = (blk >= 0) & (blk < NB)
        if not live.all():
            status |= BAD_BLOCK
        j, blk = j[live], blk[live]
        if not len(j):
            continue
        k = np.repeat(key_cache[blk, j % BS], G, axis=1)     # [n, Hq, D]
        v = np.repeat(value_cache[blk, j % BS], G, axis=1)
        x = q[lo:hi]
        s = scale * np.einsum("thd,nhd->thn", x, k)
        m = s.max(-1, keepdims=True)
        w = np.exp(s - m)
        total = w.sum(-1, keepdims=True)
        out[lo:hi] = np.einsum("thn,nhd->thd", w / total, v)
        size[lo:hi] = np.einsum("thn,nhd->thd", w / total, np.abs(v))
        lse[lo:hi] = (m + np.log(total))[..., 0]
        reach[lo:hi] = (abs(scale) * np.einsum("thd,nhd->thn", np.abs(x), np.abs(k))).max(-1)
    return out, lse, size, reach, status
