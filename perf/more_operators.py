"""Timed cases of the operators around the paged cache of a decoder with normed queries and
keys, sliding windows and requests that share what they read.

Four operators that stand beside the paged attention, append and schedule calls:

* ``norm``   - queries and keys normed for each head, rotated, written with V into the pool;
* ``window`` - causal attention over the paged cache with a sliding window, and a few first
  tokens that stay visible (bfloat16 too, and without a window);
* ``prefix`` - causal attention of requests whose first tokens lie in the same blocks: what
  they share is read and multiplied once for all of them;
* ``fork``   - rows of the block table copied, reordered and freed, with the partly filled
  block of each copy in every layer's cache.

``run`` computes a case in plain torch operations (``own`` false) or through this
package's entry points (``own`` true). ``exact`` states each operator's definition in
64 bits (whole numbers: row by row on the host).
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 64 requests: packed rows, one position a token
        {"name": "norm_decode", "op": "norm", "tokens": 64, "num_heads": 32, "kv_heads": 8,
         "head_size": 128, "rotary_dim": 128, "axes": 1, "interleaved": False,
         "block_size": 16, "dtype": "f16", "table": "f16", "weight": "f16", "packed": True,
         "positions": 8192, "pad": 0, "mix": 1},
        # a chunk of prompts of text and video, bfloat16 with 32-bit tables
        {"name": "norm_prompt", "op": "norm", "tokens": 32768, "num_heads": 32,
         "kv_heads": 8, "head_size": 128, "rotary_dim": 128, "axes": 3,
         "interleaved": False, "block_size": 32, "dtype": "bf16", "table": "f32",
         "weight": "bf16", "packed": False, "positions": 32768, "pad": 0, "mix": 2},
        # half of each head rotated, pairs side by side, an odd number of tokens and padding
        {"name": "norm_partial", "op": "norm", "tokens": 4097, "num_heads": 12,
         "kv_heads": 4, "head_size": 64, "rotary_dim": 32, "axes": 1, "interleaved": True,
         "block_size": 16, "dtype": "f16", "table": "f32", "weight": "f32", "packed": True,
         "positions": 4096, "pad": 31, "mix": 3},
        # two requests that decode with a short window: nothing but latency
        {"name": "window_tiny", "op": "window", "batch": 2, "queries": 1, "past": 400,
         "least_past": 100, "window": 128, "sinks": 4, "num_heads": 4, "kv_heads": 2,
         "head_size": 64, "block_size": 16, "dtype": "f16", "mix": 4},
        # a decode step of 64 requests, contexts of 512 to 8192, half of that visible
        {"name": "window_decode", "op": "window", "batch": 64, "queries": 1, "past": 8191,
         "least_past": 511, "window": 4096, "sinks": 4, "num_heads": 32, "kv_heads": 8,
         "head_size": 128, "block_size": 16, "dtype": "bf16", "mix": 5},
        # eight prompts of up to 2048 tokens behind up to 2048 earlier ones
        {"name": "window_prompt", "op": "window", "batch": 8, "queries": 2048, "past": 2048,
         "least_past": 0, "window": 1024, "sinks": 16, "num_heads": 32, "kv_heads": 8,
         "head_size": 128, "block_size": 32, "dtype": "bf16", "mix": 6},
        # four samples of one short prompt
        {"name": "prefix_tiny", "op": "prefix", "groups": 1, "width": 4, "shared": 500,
         "own_past": 60, "queries": 1, "num_heads": 4, "kv_heads": 2, "head_size": 64,
         "block_size": 16, "dtype": "f16", "mix": 7},
        # a decode step of 64 requests behind one system prompt of 8192 tokens
        {"name": "prefix_decode", "op": "prefix", "groups": 1, "width": 64, "shared": 8192,
         "own_past": 512, "queries": 1, "num_heads": 32, "kv_heads": 8, "head_size": 128,
         "block_size": 16, "dtype": "f16", "mix": 8},
        # questions of up to 256 tokens about two documents, eight about each
        {"name": "prefix_prompt", "op": "prefix", "groups": 2, "width": 8, "shared": 8000,
         "own_past": 0, "queries": 256, "num_heads": 32, "kv_heads": 8, "head_size": 128,
         "block_size": 32, "dtype": "bf16", "mix": 9},
        # the beams of one request change places, one layer
        {"name": "fork_tiny", "op": "fork", "groups": 1, "width": 4, "past": 400, "beams": True,
         "ends": 0.0, "block_size": 16, "max_blocks": 32, "layers": 1, "kv_heads": 2,
         "head_size": 64, "dtype": "f16", "spare": 16, "short_by": 0, "mix": 10},
        # 16 requests of four beams each, 16 layers
        {"name": "fork_beams", "op": "fork", "groups": 16, "width": 4, "past": 2000,
         "beams": True, "ends": 0.1, "block_size": 16, "max_blocks": 130, "layers": 16,
         "kv_heads": 8, "head_size": 128, "dtype": "f16", "spare": 100, "short_by": 0,
         "mix": 11},
        # a large batch: 64 prompts, each of them sampled 16 times from here on, blocks of 64,
        # a pool too small for the last ones
        {"name": "fork_samples", "op": "fork", "groups": 64, "width": 16, "past": 4000,
         "beams": False, "ends": 0.0, "block_size": 64, "max_blocks": 128, "layers": 8,
         "kv_heads": 8, "head_size": 128, "dtype": "bf16", "spare": 1000, "short_by": 20,
         "mix": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "window", "prefix", "fork"])
    mix = rng.randrange(1000, 1000000)
    dtype = rng.choice(["f16", "bf16"])
    hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    bs = rng.choice([8, 16, 32, 64])
    if op == "norm":
        return {"op": op, "tokens": _log(rng, 1, 32768),
                "num_heads": hkv * rng.choice([1, 2, 3, 4]), "kv_heads": hkv,
                "head_size": d, "rotary_dim": rng.choice([d, d, d // 2]),
                "axes": rng.choice([1, 1, 3]), "interleaved": rng.random() < 0.3,
                "block_size": bs, "dtype": dtype, "table": rng.choice([dtype, "f32"]),
                "weight": rng.choice([dtype, "f32"]), "packed": rng.random() < 0.5,
                "positions": rng.choice([8192, 32768]),
                "pad": rng.choice([0, rng.randrange(1, 100)]), "mix": mix}
    if op == "fork":
        width, past = rng.choice([2, 4, 8, 16]), _log(rng, 20, 4000)
        return {"op": op, "groups": _log(rng, 1, 32), "width": width, "past": past,
                "beams": rng.random() < 0.5, "ends": rng.choice([0.0, 0.1]),
                "block_size": bs, "max_blocks": -(-past // bs) + rng.randrange(1, 9),
                "layers": rng.choice([1, 2, 4, 8]), "kv_heads": hkv, "head_size": d,
                "dtype": dtype, "spare": _log(rng, 10, 500),
                "short_by": rng.choice([0, 0, rng.randrange(1, 10)]), "mix": mix}
    g = rng.choice([1, 2, 3, 4, 8]) if hkv < 8 else rng.choice([1, 2, 3, 4])
    heads = {"num_heads": hkv * g, "kv_heads": hkv, "head_size": d, "block_size": bs,
             "dtype": dtype, "mix": mix}
    few = rng.random() < 0.5
    if op == "window":
        shape = {"op": op, "window": rng.choice([0, _log(rng, 16, 4096), _log(rng, 16, 4096)]),
                 "sinks": rng.choice([0, 1, 4, 64, 130])}
        if few:   # single tokens (or a few, where drafts are checked)
            return {**shape, "batch": _log(rng, 1, 64), "queries": rng.choice([1, 1, 1, 4]),
                    "past": _log(rng, 64, 8000), "least_past": rng.choice([0, 50]), **heads}
        return {**shape, "batch": _log(rng, 1, 8), "queries": _log(rng, 8, 2048),
                "past": _log(rng, 1, 2048), "least_past": 0, **heads}
    groups = rng.choice([1, 1, 2, 3])
    if few:
        return {"op": op, "groups": groups, "width": _log(rng, 2, 64 // groups),
                "shared": _log(rng, 40, 8192), "own_past": _log(rng, 1, 512),
                "queries": rng.choice([1, 1, 4]), **heads}
    return {"op": op, "groups": groups, "width": rng.choice([1, 2, 3, 5]),
            "shared": _log(rng, 40, 8000), "own_past": rng.choice([0, _log(rng, 1, 256)]),
            "queries": _log(rng, 8, 256), **heads}


# ------------------------------------------------------------------------- lengths, work
def _ceil(a, b):
    return -(-a // b)


def _window_lengths(case):
    """New and earlier tokens of each request."""
    r = random.Random(case["mix"])
    new, past = [], []
    for _ in range(case["batch"]):
        new.append(case["queries"] if case["queries"] <= 8 else r.randrange(1, case["queries"] + 1))
        past.append(r.randrange(case["least_past"], max(case["least_past"], case["past"]) + 1))
    return new, past


def _prefix_lengths(case):
    """The shared tokens of each group, then each request's new and earlier tokens."""
    r = random.Random(case["mix"])
    shared, new, past = [], [], []
    for _ in range(case["groups"]):
        n = r.randrange(max(1, 3 * case["shared"] // 4), case["shared"] + 1) \
            if case["groups"] > 1 else case["shared"]
        shared.append(n)
        for _ in range(case["width"]):
            new.append(case["queries"] if case["queries"] <= 8
                       else r.randrange(1, case["queries"] + 1))
            past.append(n + r.randrange(case["own_past"] + 1))
    return shared, new, past


def _fork_rows(case):
    """Lengths, parents and (for the blocks) the tokens that a group's rows share."""
    r = random.Random(case["mix"])
    w, past, parents, prompts = case["width"], [], [], []
    for g in range(case["groups"]):
        prompt = r.randrange(1, case["past"] // 2 + 2)
        prompts.append(prompt)
        n = r.randrange(prompt, case["past"] + 1)
        ends = r.random() < case["ends"]
        for x in range(w):
            past.append(n if case["beams"] or x == 0 else 0)
            at = g * w + (r.randrange(w) if case["beams"] else 0)
            parents.append(-1 if ends else at)
    return past, parents, prompts


def _fork_plan(past, parents, block_size):
    """For each row the length it takes over, and whether it needs a block of its own."""
    keeper = {}
    for b, p in enumerate(parents):
        if p >= 0 and (p not in keeper or b == p):
            keeper[p] = b
    return [(past[p], keeper[p] != b and past[p] % block_size > 0) if p >= 0 else (0, False)
            for b, p in enumerate(parents)]


def _seen(pos, window, sinks):
    """Keys that the token at this position sees."""
    if window <= 0 or pos < window:
        return pos + 1
    return window + min(sinks, pos + 1 - window)


def work(case):
    d, hkv = case["head_size"], case["kv_heads"]
    if case["op"] == "norm":
        t, r = case["tokens"], case["rotary_dim"]
        rows = case["num_heads"] + 2 * hkv
        size, wsize = (4 if case[k] == "f32" else 2 for k in ("table", "weight"))
        tables = 2 * size * (r // 2) * min(t, case["positions"])
        return {"bytes": 4 * t * rows * d + 4 * t * (case["axes"] + 1) + tables + 2 * wsize * d,
                "flops": t * (case["num_heads"] + hkv) * (4 * d + 3 * r)}
    if case["op"] == "fork":
        past, parents, _ = _fork_rows(case)
        bs, rows = case["block_size"], len(past)
        parts = [n % bs for n, fresh in _fork_plan(past, parents, bs) if fresh]
        if case["short_by"] > 0 and not case["beams"] and case["ends"] == 0:
            parts = parts[:-case["short_by"]]      # the pool has no blocks for the last ones
        copied = sum(parts) * 2 * case["layers"] * hkv * d * 2
        held = sum(_ceil(past[p], bs) for p in set(parents) if p >= 0)
        return {"bytes": 2 * copied + 4 * (held + rows * case["max_blocks"] + 3 * rows + 1),
                "flops": 0}
    hq = case["num_heads"]
    if case["op"] == "window":
        new, past = _window_lengths(case)
        w, s = case["window"], case["sinks"]
        keys = [_seen(p + n - 1, w + n - 1 if w else 0, s) for n, p in zip(new, past)]
        pairs = sum(_seen(p + i, w, s) for n, p in zip(new, past) for i in range(n))
    else:
        shared, new, past = _prefix_lengths(case)
        of = [g for g in range(case["groups"]) for _ in range(case["width"])]
        keys = shared + [p + n - shared[g] for g, n, p in zip(of, new, past)]
        pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
    return {"bytes": 4 * sum(new) * hq * d + 4 * sum(new) * hq + 4 * sum(keys) * hkv * d
            + 4 * sum(_ceil(k, case["block_size"]) for k in keys), "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------------------- inputs
def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _gen(seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return gen


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _prepare_norm(case, seed):
    gen, rng = _gen(seed), np.random.default_rng(seed)
    t, hq, hkv, d = case["tokens"], case["num_heads"], case["kv_heads"], case["head_size"]
    dt, bs = _TYPES[case["dtype"]], case["block_size"]
    rows = t + case["pad"]
    if case["packed"]:
        q, k, v = _normal(gen, (rows, (hq + 2 * hkv) * d), dt), None, None
    else:
        q, k, v = (_normal(gen, (rows, h * d), dt) for h in (hq, hkv, hkv))
    blocks = _ceil(t, bs) + 8
    order = rng.permutation(blocks)
    i = np.arange(t)
    slots = np.full(rows, -1, np.int32)
    slots[:t] = order[i // bs] * bs + i % bs
    # runs of tokens, one for each request; frames, rows and columns step at their own pace
    pos = np.zeros((case["axes"], rows), np.int64)
    for a in range(case["axes"]):
        pos[a] = rng.integers(0, case["positions"]) + np.arange(rows) // (1, 7, 3)[a]
    half = case["rotary_dim"] // 2
    turn = 10000.0 ** (-np.arange(half, dtype=np.float64) / half)
    angle = torch.from_numpy(np.arange(case["positions"], dtype=np.float64)[:, None] * turn)
    tt, wt = _TYPES[case["table"]], _TYPES[case["weight"]]
    axis = [a * case["axes"] // half for a in range(half)]
    weight = lambda: (1 + 0.2 * _normal(gen, (d,), torch.float32)).to(wt)  # noqa: E731
    return {"q": q, "k": k, "v": v, "slots": _dev(slots),
            "pos": _dev((pos % case["positions"]).astype(np.int32)),
            "cos": torch.cos(angle).to(tt).to(DEV), "sin": torch.sin(angle).to(tt).to(DEV),
            "axis": axis, "axis_dev": _dev(np.array(axis, np.int64)),
            "qw": weight(), "kw": weight(), "eps": 1e-6,
            "kc": _normal(gen, (blocks, bs, hkv, d), dt),
            "vc": _normal(gen, (blocks, bs, hkv, d), dt),
            "q_out": torch.zeros((rows, hq * d), dtype=dt, device=DEV),
            "hq": hq, "hkv": hkv, "d": d, "half": half, "interleaved": case["interleaved"]}


def _attention_state(case, seed, new, past, table, num_blocks):
    gen = _gen(seed)
    hq, hkv, d, dt = case["num_heads"], case["kv_heads"], case["head_size"], _TYPES[case["dtype"]]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    t, pool = int(cu[-1]), (num_blocks, case["block_size"], hkv, d)
    return {"q": _normal(gen, (t, hq * d), dt), "kc": _normal(gen, pool, dt),
            "vc": _normal(gen, pool, dt), "cu": _dev(cu), "table": _dev(table),
            "past": _dev(np.array(past, np.int32)), "hq": hq, "hkv": hkv, "d": d,
            "bs": case["block_size"], "max_q": max(new), "max_k": max(n + p for n, p in
                                                                      zip(new, past)),
            "window": 0, "sinks": 0, "out": torch.zeros((t, hq * d), dtype=dt, device=DEV),
            "lse": torch.zeros((t, hq), dtype=torch.float32, device=DEV)}


def _prepare_window(case, seed):
    new, past = _window_lengths(case)
    bs, w = case["block_size"], case["window"]
    need = [_ceil(n + p, bs) for n, p in zip(new, past)]
    ids = np.random.default_rng(seed).permutation(sum(need) + 16).astype(np.int32)
    table, at = np.full((case["batch"], max(need)), -1, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
        if w > 0:   # blocks that no token sees any more were given back
            first, last = _ceil(case["sinks"], bs), max(0, past[b] - w + 1) // bs
            table[b, first:max(first, last)] = -1
    s = _attention_state(case, seed, new, past, table, len(ids))
    s["window"], s["sinks"] = w, case["sinks"]
    return s


def _prepare_prefix(case, seed):
    shared, new, past = _prefix_lengths(case)
    bs, width = case["block_size"], case["width"]
    lead = [n // bs for n in shared]       # whole blocks that a group's rows have in common
    need = [_ceil(n + p, bs) - lead[b // width] for b, (n, p) in enumerate(zip(new, past))]
    ids = np.random.default_rng(seed).permutation(sum(lead) + sum(need) + 16).astype(np.int32)
    table, at = np.full((len(new), max(_ceil(n + p, bs) for n, p in zip(new, past))), -1,
                        np.int32), 0
    for g, n in enumerate(lead):
        table[g * width:(g + 1) * width, :n] = ids[at:at + n]
        at += n
    for b, n in enumerate(need):
        table[b, lead[b // width]:lead[b // width] + n] = ids[at:at + n]
        at += n
    s = _attention_state(case, seed, new, past, table, len(ids))
    s["groups"] = _dev(np.arange(0, len(new) + 1, width, dtype=np.int32))
    s["shared"] = _dev(np.array([n * bs for n in lead], np.int32))
    return s


def _prepare_fork(case, seed):
    past, parents, prompts = _fork_rows(case)
    bs, mb, w = case["block_size"], case["max_blocks"], case["width"]
    need = [_ceil(n, bs) for n in past]
    fresh = sum(f for _, f in _fork_plan(past, parents, bs))
    table = np.full((len(past), mb), -1, np.int64)
    at = 0
    for b, n in enumerate(need):           # the beams of a request share its prompt's blocks
        lead = prompts[b // w] // bs if case["beams"] and b % w > 0 else 0
        table[b, :lead] = table[b - b % w, :lead]
        table[b, lead:n] = np.arange(at, at + n - lead)
        at += n - lead
    num_blocks = at + max(fresh + 8, case["spare"])
    if case["short_by"] > 0 and case["ends"] == 0:
        num_blocks = at + max(0, fresh - case["short_by"])
    ids = np.random.default_rng(seed).permutation(num_blocks)
    table = np.where(table >= 0, ids[np.maximum(table, 0)], -1).astype(np.int32)
    shape = (2 * case["layers"], num_blocks, bs, case["kv_heads"], case["head_size"])
    pool = torch.randn(shape, generator=_gen(seed), device=DEV, dtype=_TYPES[case["dtype"]])
    i32 = dict(dtype=torch.int32, device=DEV)
    return {"pool": pool, "caches": list(pool.unbind(0)), "table": _dev(table),
            "past": _dev(np.array(past, np.int32)), "parents": _dev(np.array(parents, np.int32)),
            "new_past": torch.zeros(len(past), **i32),
            "new_table": torch.zeros((len(past), mb), **i32), "free": torch.zeros(1, **i32)}


def prepare(case, seed):
    s = {"norm": _prepare_norm, "window": _prepare_window, "prefix": _prepare_prefix,
         "fork": _prepare_fork}[case["op"]](case, seed)
    s["op"] = case["op"]
    return s


# ---------------------------------------------------------------------------- plain forms
def _plain_norm(s):
    hq, hkv, d, half = s["hq"], s["hkv"], s["d"], s["half"]
    if s["k"] is None:
        q, k, v = s["q"].split([hq * d, hkv * d, hkv * d], dim=1)
    else:
        q, k, v = s["q"], s["k"], s["v"]
    n = q.shape[0]
    at = s["pos"].long()[s["axis_dev"]].t()                      # [tokens, pairs]
    pair = torch.arange(half, device=DEV)
    c, w = s["cos"].float()[at, pair][:, None], s["sin"].float()[at, pair][:, None]

    def turned(x, heads, weight):
        x = x.reshape(n, heads, d).float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight.float()
        if s["interleaved"]:
            a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
            r = torch.stack([a * c - b * w, b * c + a * w], -1).flatten(2)
        else:
            a, b = x[..., :half], x[..., half:2 * half]
            r = torch.cat([a * c - b * w, b * c + a * w], -1)
        return torch.cat([r, x[..., 2 * half:]], -1).to(s["q"].dtype)

    live = s["slots"] >= 0
    to = s["slots"][live].long()
    s["q_out"][live] = turned(q, hq, s["qw"]).flatten(1)[live]
    s["kc"].view(-1, hkv, d)[to] = turned(k, hkv, s["kw"])[live]
    s["vc"].view(-1, hkv, d)[to] = v.reshape(n, hkv, d)[live]


def _plain_attention(s):
    """Causal attention of every request over its own row of the table, padded to the longest:
    the window and the sinks are a mask."""
    hq, hkv, d, bs = s["hq"], s["hkv"], s["d"], s["bs"]
    g, b, mq, mk = hq // hkv, s["past"].numel(), s["max_q"], s["max_k"]
    cu = s["cu"].long()
    i = torch.arange(s["q"].shape[0], device=DEV)
    of = torch.searchsorted(cu[1:], i, right=True)
    q = torch.zeros((b, mq, hq * d), dtype=torch.float32, device=DEV)
    q[of, i - cu[of]] = s["q"].float()
    q = q.view(b, mq, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * mq, d)
    j = torch.arange(mk, device=DEV)
    block = s["table"].long()[:, j // bs]
    row = torch.where(block >= 0, block * bs + j % bs, torch.zeros_like(block))
    k = s["kc"].view(-1, hkv, d)[row].float().permute(0, 2, 3, 1)   # [b, hkv, d, mk]
    v = s["vc"].view(-1, hkv, d)[row].float().permute(0, 2, 1, 3)
    p = torch.matmul(q * (1.0 / math.sqrt(d)), k)
    pos = s["past"].long()[:, None] + torch.arange(mq, device=DEV)  # [b, mq]
    unseen = j > pos[..., None]
    if s["window"] > 0:
        unseen |= (j <= pos[..., None] - s["window"]) & (j >= s["sinks"])
    p.view(b, hkv, g, mq, mk).masked_fill_(unseen[:, None, None], float("-inf"))
    top = p.amax(-1, keepdim=True)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / total
    o = o.view(b, hkv, g, mq, d).permute(0, 3, 1, 2, 4).reshape(b, mq, hq * d)
    lse = (top + torch.log(total)).view(b, hkv, g, mq).permute(0, 3, 1, 2).reshape(b, mq, hq)
    s["out"].copy_(o[of, i - cu[of]])
    s["lse"].copy_(lse[of, i - cu[of]])


def _plain_fork(s):
    table, past, parents = s["table"].long(), s["past"].long(), s["parents"].long()
    rows, mb = table.shape
    num_blocks, bs = s["pool"].shape[1:3]
    row, live = torch.arange(rows, device=DEV), parents >= 0
    of = parents.clamp(min=0)
    # the row that keeps a parent's last block: the parent itself, or the first of its copies
    rank = torch.where(live, torch.where(of == row, torch.full_like(row, -1), row),
                       torch.full_like(row, rows))
    best = torch.full_like(row, rows).scatter_reduce(0, of, rank, "amin")
    n = torch.where(live, past[of], torch.zeros_like(past))
    fresh = live & (n % bs > 0) & (best[of] != rank)
    col = torch.arange(mb, device=DEV)
    held = (n + bs - 1) // bs - fresh.long()
    new = torch.where(col[None, :] < held[:, None], table[of], torch.full_like(table, -1))
    taken = torch.zeros(num_blocks, dtype=torch.int64, device=DEV)
    taken[new[new >= 0]] = 1
    free = torch.nonzero(taken == 0)[:, 0]
    nth = torch.cumsum(fresh.long(), 0) - 1
    ok = fresh & (nth < free.numel())
    dst, src = free[nth[ok]], table[of[ok], n[ok] // bs]
    new[row[ok], n[ok] // bs] = dst
    lost = fresh & ~ok
    new[lost], n[lost] = -1, 0
    at = torch.arange(bs, device=DEV)
    part = at[None, :] < (n[ok] % bs)[:, None]
    pool = s["pool"].view(s["pool"].shape[0], num_blocks * bs, -1)
    pool[:, (dst[:, None] * bs + at)[part]] = pool[:, (src[:, None] * bs + at)[part]]
    s["new_table"].copy_(new)
    s["new_past"].copy_(n)
    s["free"].copy_(free.numel() - ok.sum())


# -------------------------------------------------------------------- the package's calls
def _own_norm(s):
    from paged_kv_cache_231_gb300 import binding as B
    B.pkv_paged_append_norm_rotary(
        s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"], s["pos"], num_heads=s["hq"],
        kv_num_heads=s["hkv"], query_weight=s["qw"], key_weight=s["kw"], epsilon=s["eps"],
        cos_cache=s["cos"], sin_cache=s["sin"], rotary_dim=2 * s["half"], pair_axis=s["axis"],
        rotary_interleaved=s["interleaved"], query_out=s["q_out"])


def _own_window(s):
    from paged_kv_cache_231_gb300 import binding as B
    B.pkv_paged_window_attention(
        s["q"], s["kc"], s["vc"], s["cu"], s["past"], s["table"], num_heads=s["hq"],
        kv_num_heads=s["hkv"], window=s["window"], sinks=s["sinks"], max_query_len=s["max_q"],
        output=s["out"], lse=s["lse"])


def _own_prefix(s):
    from paged_kv_cache_231_gb300 import binding as B
    B.pkv_paged_prefix_attention(
        s["q"], s["kc"], s["vc"], s["cu"], s["past"], s["table"], s["groups"], s["shared"],
        num_heads=s["hq"], kv_num_heads=s["hkv"], max_query_len=s["max_q"], output=s["out"],
        lse=s["lse"])


def _own_fork(s):
    from paged_kv_cache_231_gb300 import binding as B
    B.pkv_paged_fork(s["parents"], s["past"], s["table"], s["caches"],
                     new_past_seqlens=s["new_past"], new_block_table=s["new_table"],
                     free_blocks=s["free"])


def run(s):
    if own:
        {"norm": _own_norm, "window": _own_window, "prefix": _own_prefix,
         "fork": _own_fork}[s["op"]](s)
    else:
        {"norm": _plain_norm, "window": _plain_attention, "prefix": _plain_attention,
         "fork": _plain_fork}[s["op"]](s)
    names = {"norm": ("q_out", "kc", "vc"), "window": ("out", "lse"), "prefix": ("out", "lse"),
             "fork": ("new_past", "new_table", "free", "pool")}[s["op"]]
    return {n: s[n] for n in names}


# ------------------------------------------------------------------------------ definition
def _exact_norm(s):
    hq, hkv, d, r = s["hq"], s["hkv"], s["d"], 2 * s["half"]
    x = s["q"] if s["k"] is None else torch.cat([s["q"], s["k"], s["v"]], 1)
    x = x.double().view(x.shape[0], hq + 2 * hkv, d).clone()
    for rows, weight in ((slice(0, hq), s["qw"]), (slice(hq, hq + hkv), s["kw"])):
        x[:, rows] *= weight.double() / torch.sqrt(
            (x[:, rows] ** 2).sum(-1, keepdim=True) / d + s["eps"])
    of = torch.arange(r, device=DEV)
    pair = of // 2 if s["interleaved"] else of % s["half"]
    first = of % 2 == 0 if s["interleaved"] else of < s["half"]
    other = of ^ 1 if s["interleaved"] else (of + s["half"]) % r
    where = s["pos"].long()[s["axis_dev"][pair]].t()
    co, si = s["cos"].double()[where, pair], s["sin"].double()[where, pair]
    mine, mate = x[:, :hq + hkv, :r], x[:, :hq + hkv, other]
    sign = torch.where(first, -1.0, 1.0).double()
    x[:, :hq + hkv, :r] = mine * co[:, None] + sign * mate * si[:, None]
    q_out, kc, vc = s["q_out"].double(), s["kc"].double(), s["vc"].double()
    live = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"][live].long()
    q_out[live] = x[live, :hq].flatten(1)
    kc.view(-1, hkv, d)[at] = x[live, hq:hq + hkv]
    vc.view(-1, hkv, d)[at] = x[live, hq + hkv:]
    return {"q_out": q_out, "kc": kc, "vc": vc}


def _exact_attention(s):
    hq, hkv, d, bs = s["hq"], s["hkv"], s["d"], s["bs"]
    cu, past, w = s["cu"].tolist(), s["past"].tolist(), s["window"]
    out = torch.zeros((cu[-1], hq, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((cu[-1], hq), dtype=torch.float64, device=DEV)
    for b, p in enumerate(past):
        q0, q1 = cu[b], cu[b + 1]
        n = p + q1 - q0
        j = torch.arange(n, device=DEV)
        pos = torch.arange(p, n, device=DEV)[:, None]
        seen = (j <= pos) & ((j > pos - w) | (j < s["sinks"])) if w > 0 else j <= pos
        keys = torch.nonzero(seen.any(0))[:, 0]       # no others are read
        at = s["table"][b].long()[keys // bs] * bs + keys % bs
        k = s["kc"].view(-1, hkv, d)[at].double().repeat_interleave(hq // hkv, 1)
        v = s["vc"].view(-1, hkv, d)[at].double().repeat_interleave(hq // hkv, 1)
        q = s["q"][q0:q1].double().view(-1, hq, d)
        score = torch.einsum("thd,nhd->htn", q, k) / math.sqrt(d)
        score = score.masked_fill(~seen[:, keys], float("-inf"))
        lse[q0:q1] = torch.logsumexp(score, -1).t()
        out[q0:q1] = torch.einsum("htn,nhd->thd", torch.softmax(score, -1), v)
    return {"out": out.flatten(1), "lse": lse}


def _exact_fork(s):
    table, past = s["table"].cpu().numpy().astype(np.int64), s["past"].tolist()
    parents, (num_blocks, bs) = s["parents"].tolist(), s["pool"].shape[1:3]
    plan = _fork_plan(past, parents, bs)
    new = np.full_like(table, -1)
    for b, (n, fresh) in enumerate(plan):
        held = _ceil(n, bs) - (1 if fresh else 0)
        new[b, :held] = table[parents[b], :held]
    taken = set(new[new >= 0].tolist())
    free = [x for x in range(num_blocks) if x not in taken]
    pool, lengths, used = s["pool"], [], 0
    for b, (n, fresh) in enumerate(plan):
        if fresh and used == len(free):
            new[b], n = -1, 0
        elif fresh:
            new[b, n // bs] = free[used]
            pool[:, free[used], :n % bs] = pool[:, int(table[parents[b], n // bs]), :n % bs]
            used += 1
        lengths.append(n)
    as32 = lambda x: torch.from_numpy(np.asarray(x, np.int32))  # noqa: E731
    return {"new_past": as32(lengths), "new_table": as32(new), "free": as32([len(free) - used]),
            "pool": pool}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "window": _exact_attention, "prefix": _exact_attention,
            "fork": _exact_fork}[case["op"]](s)
