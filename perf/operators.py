"""Timed cases of the step operators of a decoder with image, video or audio inputs.

Three operators that stand beside the paged attention call:

* ``schedule`` - block tables, slot maps and cumulative lengths from request lengths;
* ``axes``     - rotary positions with several axes, written with K and V into the pool;
* ``cross``    - attention of ragged queries over an encoder's states in a paged pool.

``run`` computes a case in plain torch operations (``own`` false) or through this
package's entry points (``own`` true). ``exact`` states each operator's definition in
64 bits (whole numbers: sequence by sequence on the host).
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
        # two requests that decode: nothing but latency
        {"name": "schedule_tiny", "op": "schedule", "batch": 2, "past": 400,
         "new": 1, "long_share": 0.0, "block_size": 16, "max_blocks": 32, "spare": 64,
         "short_by": 0, "pad": 0, "mix": 1},
        # one decode step of 64 requests, contexts of 512 to 8192 keys in blocks of 16
        {"name": "schedule_decode", "op": "schedule", "batch": 64, "past": 8192,
         "new": 1, "long_share": 0.0, "block_size": 16, "max_blocks": 520, "spare": 4096,
         "short_by": 0, "pad": 0, "mix": 2},
        # half of 16 requests prefill up to 2048 tokens, half decode; blocks of 32
        {"name": "schedule_mixed", "op": "schedule", "batch": 16, "past": 4096,
         "new": 2048, "long_share": 0.5, "block_size": 32, "max_blocks": 200, "spare": 512,
         "short_by": 0, "pad": 61, "mix": 3},
        # a full pool: 2048 rows, a third of them taking in prompts of up to 1000 tokens,
        # and a pool too small for the last of them
        {"name": "schedule_full", "op": "schedule", "batch": 2048, "past": 8192,
         "new": 1000, "long_share": 0.33, "block_size": 16, "max_blocks": 600, "spare": 0,
         "short_by": 700, "pad": 513, "mix": 4},
        # one decode step of 64 requests whose prompts held images: packed rows
        {"name": "axes_decode", "op": "axes", "tokens": 64, "num_heads": 32, "kv_heads": 8,
         "head_size": 128, "rotary_dim": 128, "axes": 3, "interleaved": False,
         "turns": False, "block_size": 16, "dtype": "f16", "table": "f16", "packed": True,
         "positions": 8192, "pad": 0, "mix": 5},
        # a chunk of video and text tokens of a prompt, bfloat16 with 32-bit tables
        {"name": "axes_video", "op": "axes", "tokens": 32768, "num_heads": 32,
         "kv_heads": 8, "head_size": 128, "rotary_dim": 128, "axes": 3,
         "interleaved": False, "turns": True, "block_size": 32, "dtype": "bf16",
         "table": "f32", "packed": False, "positions": 32768, "pad": 0, "mix": 6},
        # image tokens with height and width only, half of each head rotated, pairs side
        # by side, an odd number of tokens
        {"name": "axes_image", "op": "axes", "tokens": 4097, "num_heads": 12,
         "kv_heads": 4, "head_size": 64, "rotary_dim": 32, "axes": 2, "interleaved": True,
         "turns": False, "block_size": 16, "dtype": "f16", "table": "f32", "packed": True,
         "positions": 4096, "pad": 31, "mix": 7},
        # a decode step of two requests over a few hundred encoder states
        {"name": "cross_tiny", "op": "cross", "batch": 2, "queries": 1, "keys": 400,
         "least_keys": 100, "num_heads": 4, "kv_heads": 2, "head_size": 64,
         "block_size": 16, "dtype": "f16", "mix": 8},
        # a decode step of 64 requests, 512 to 8192 states each
        {"name": "cross_decode", "op": "cross", "batch": 64, "queries": 1, "keys": 8192,
         "least_keys": 512, "num_heads": 32, "kv_heads": 8, "head_size": 128,
         "block_size": 16, "dtype": "f16", "mix": 9},
        # a decode step of 128 requests over up to 1500 audio frames, one query head to a
        # kv head, bfloat16; some encoders have not answered yet (no states)
        {"name": "cross_audio", "op": "cross", "batch": 128, "queries": 1, "keys": 1500,
         "least_keys": 0, "num_heads": 16, "kv_heads": 16, "head_size": 64,
         "block_size": 32, "dtype": "bf16", "mix": 10},
        # prompts of up to 2048 tokens over up to 4096 image states
        {"name": "cross_prompt", "op": "cross", "batch": 16, "queries": 2048, "keys": 4096,
         "least_keys": 1, "num_heads": 32, "kv_heads": 8, "head_size": 128,
         "block_size": 32, "dtype": "f16", "mix": 11},
        # two questions of up to a hundred tokens about long videos
        {"name": "cross_question", "op": "cross", "batch": 2, "queries": 100, "keys": 60000,
         "least_keys": 20000, "num_heads": 16, "kv_heads": 16, "head_size": 64,
         "block_size": 64, "dtype": "bf16", "mix": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["schedule", "axes", "cross"])
    mix = rng.randrange(1000, 1000000)
    if op == "schedule":
        past, bs = _log(rng, 200, 8192), rng.choice([16, 24, 32, 64])
        batch = _log(rng, 1, 2048)
        new = rng.choice([1, 1, rng.randrange(2, 9), _log(rng, 16, 1000)])
        return {"op": op, "batch": batch, "past": past, "new": new,
                "long_share": rng.choice([0.1, 0.33, 0.33 if batch > 512 else 1.0]),
                "block_size": bs, "max_blocks": -(-(past + new) // bs) + rng.randrange(9),
                "spare": rng.choice([0, _log(rng, 10, 5000)]),
                "short_by": rng.choice([0, 0, rng.randrange(1, 50)]),
                "pad": rng.choice([0, rng.randrange(1, 200)]), "mix": mix}
    if op == "axes":
        hkv = rng.choice([1, 2, 4, 8])
        d = rng.choice([64, 128])
        dtype = rng.choice(["f16", "bf16"])
        return {"op": op, "tokens": _log(rng, 1, 32768),
                "num_heads": hkv * rng.choice([1, 2, 3, 4]), "kv_heads": hkv,
                "head_size": d, "rotary_dim": rng.choice([d, d, d // 2]),
                "axes": rng.choice([1, 2, 3, 3]), "interleaved": rng.random() < 0.3,
                "turns": rng.random() < 0.3, "block_size": rng.choice([8, 16, 32, 64]),
                "dtype": dtype, "table": rng.choice([dtype, "f32"]),
                "packed": rng.random() < 0.5, "positions": rng.choice([8192, 32768]),
                "pad": rng.choice([0, rng.randrange(1, 100)]), "mix": mix}
    d, bs = rng.choice([64, 128]), rng.choice([8, 16, 32, 64])
    dtype = rng.choice(["f16", "bf16"])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 8])
    if rng.random() < 0.5:   # single tokens (or a few, where drafts are checked)
        return {"op": op, "batch": _log(rng, 1, 64), "queries": rng.choice([1, 1, 1, 4]),
                "keys": _log(rng, 64, 8192), "least_keys": rng.choice([0, 1, 60]),
                "num_heads": hkv * g, "kv_heads": hkv, "head_size": d, "block_size": bs,
                "dtype": dtype, "mix": mix}
    return {"op": op, "batch": _log(rng, 1, 16), "queries": _log(rng, 8, 2048),
            "keys": _log(rng, 64, 4096), "least_keys": rng.choice([0, 1, 60]),
            "num_heads": hkv * min(g, 4), "kv_heads": hkv, "head_size": d,
            "block_size": bs, "dtype": dtype, "mix": mix}


# ------------------------------------------------------------------------- lengths, work
def _schedule_lengths(case):
    """Lengths of the rows: a share of them take in many tokens, the others one each; one
    row in sixteen idles (no new token), where there are that many."""
    r = random.Random(case["mix"])
    past, new = [], []
    for b in range(case["batch"]):
        long = r.random() < case["long_share"]
        past.append(0 if long and r.random() < 0.5 else r.randrange(min(1, case["past"]), case["past"] + 1))
        new.append(0 if b % 16 == 13 else r.randrange(1, case["new"] + 1) if long or case["long_share"] == 0 else 1)
    return past, new


def _cross_lengths(case):
    """Queries and states of each request; where there may be none, one in sixteen has no
    states."""
    r = random.Random(case["mix"])
    nq, nk = [], []
    for b in range(case["batch"]):
        nq.append(case["queries"] if case["queries"] <= 8 else r.randrange(1, case["queries"] + 1))
        n = r.randrange(case["least_keys"], max(case["least_keys"], case["keys"]) + 1)
        nk.append(0 if case["least_keys"] == 0 and b % 16 == 5 else n)
    return nq, nk


def _ceil(a, b):
    return -(-a // b)


def work(case):
    if case["op"] == "schedule":
        past, new = _schedule_lengths(case)
        bs = case["block_size"]
        tokens = sum(new) + case["pad"]
        held = sum(_ceil(p, bs) for p in past)
        fresh = sum(_ceil(p + n, bs) - _ceil(p, bs) for p, n in zip(past, new))
        rows = case["batch"]
        # lengths, held entries; new entries, slots, positions, cumulative and total lengths
        return {"bytes": 4 * (2 * rows + held + fresh + 2 * tokens + 2 * rows + 2), "flops": 0}
    if case["op"] == "axes":
        t, d, r = case["tokens"], case["head_size"], case["rotary_dim"]
        rows = case["num_heads"] + 2 * case["kv_heads"]
        size = 4 if case["table"] == "f32" else 2
        tables = 2 * size * (r // 2) * min(t, case["positions"])
        return {"bytes": 4 * t * rows * d + 4 * t * (case["axes"] + 1) + tables,
                "flops": 3 * t * (case["num_heads"] + case["kv_heads"]) * r}
    nq, nk = _cross_lengths(case)
    d, hq, hkv, bs = case["head_size"], case["num_heads"], case["kv_heads"], case["block_size"]
    pairs = sum(a * b for a, b in zip(nq, nk))
    return {"bytes": 4 * sum(nq) * hq * d + 4 * sum(nq) * hq + 4 * sum(nk) * hkv * d
            + 4 * sum(_ceil(b, bs) for b in nk), "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------------------- inputs
def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _prepare_schedule(case, seed):
    past, new = _schedule_lengths(case)
    bs, mb = case["block_size"], case["max_blocks"]
    held = [_ceil(p, bs) for p in past]
    fresh = sum(_ceil(p + n, bs) - h for p, n, h in zip(past, new, held))
    num_blocks = max(1, sum(held) + fresh + case["spare"] - min(case["short_by"], fresh))
    ids = np.random.default_rng(seed).permutation(num_blocks).astype(np.int32)
    table = np.full((case["batch"], mb), -1, np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = ids[at:at + h]
        at += h
    tokens = sum(new) + case["pad"]
    i32 = dict(dtype=torch.int32, device=DEV)
    return {"past": _dev(np.array(past, np.int32)), "new": _dev(np.array(new, np.int32)),
            "table": _dev(table), "num_blocks": num_blocks, "block_size": bs,
            "tokens": tokens, "cu": torch.zeros(case["batch"] + 1, **i32),
            "slots": torch.zeros(tokens, **i32), "positions": torch.zeros(tokens, **i32),
            "total": torch.zeros(case["batch"], **i32), "free": torch.zeros(1, **i32)}


def _axis_positions(rng, tokens, axes, positions):
    """Positions of a prompt: runs of text, where all axes step together, and grids of
    frames, rows and columns that start where the text ended."""
    out = np.zeros((axes, tokens), np.int64)
    at = start = 0
    while at < tokens:
        n = min(tokens - at, int(rng.integers(1, 200)))
        out[:, at:at + n] = start + np.arange(n)
        at, start = at + n, start + n
        if at < tokens:
            f, h, w = int(rng.integers(1, 9)), int(rng.integers(2, 40)), int(rng.integers(2, 40))
            grid = np.stack(np.meshgrid(np.arange(f), np.arange(h), np.arange(w), indexing="ij"))
            n = min(tokens - at, f * h * w)
            out[:, at:at + n] = start + grid.reshape(3, -1)[3 - axes:, :n]
            at, start = at + n, start + max(f, h, w)
    return out % positions


def _axis_of_pair(case):
    """Which axis turns each pair: sections one after the other, or the axes by turns."""
    pairs, axes = case["rotary_dim"] // 2, case["axes"]
    if case["turns"]:
        return [i % axes for i in range(pairs)]
    first = pairs - (axes - 1) * (3 * pairs // (4 * axes)) if axes > 1 else pairs
    rest = 3 * pairs // (4 * axes)
    return [0 if i < first else 1 + (i - first) // rest for i in range(pairs)]


def _prepare_axes(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
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
    pos = np.zeros((case["axes"], rows), np.int32)
    pos[:, :t] = _axis_positions(rng, t, case["axes"], case["positions"])
    half = case["rotary_dim"] // 2
    turn = 10000.0 ** (-np.arange(half, dtype=np.float64) / half)
    angle = torch.from_numpy(np.arange(case["positions"], dtype=np.float64)[:, None] * turn)
    tt = _TYPES[case["table"]]
    axis = _axis_of_pair(case)
    return {"q": q, "k": k, "v": v, "slots": _dev(slots), "pos": _dev(pos),
            "cos": torch.cos(angle).to(tt).to(DEV), "sin": torch.sin(angle).to(tt).to(DEV),
            "axis": axis, "axis_dev": _dev(np.array(axis, np.int64)),
            "kc": _normal(gen, (blocks, bs, hkv, d), dt),
            "vc": _normal(gen, (blocks, bs, hkv, d), dt),
            "q_out": torch.zeros((rows, hq * d), dtype=dt, device=DEV),
            "hq": hq, "hkv": hkv, "d": d, "half": half, "interleaved": case["interleaved"]}


def _prepare_cross(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    nq, nk = _cross_lengths(case)
    bs, hq, hkv, d = case["block_size"], case["num_heads"], case["kv_heads"], case["head_size"]
    dt = _TYPES[case["dtype"]]
    need = [_ceil(n, bs) for n in nk]
    num_blocks = sum(need) + 16
    ids = np.random.default_rng(seed).permutation(num_blocks).astype(np.int32)
    mb = max(max(need), 1)
    table = np.full((case["batch"], mb), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    cu = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    t = int(cu[-1])
    return {"q": _normal(gen, (t, hq * d), dt), "kc": _normal(gen, (num_blocks, bs, hkv, d), dt),
            "vc": _normal(gen, (num_blocks, bs, hkv, d), dt), "cu": _dev(cu),
            "nk": _dev(np.array(nk, np.int32)), "table": _dev(table), "hq": hq, "hkv": hkv,
            "d": d, "bs": bs, "max_q": max(nq), "max_k": max(max(nk), 1),
            "out": torch.zeros((t, hq * d), dtype=dt, device=DEV),
            "lse": torch.zeros((t, hq), dtype=torch.float32, device=DEV)}


def prepare(case, seed):
    s = {"schedule": _prepare_schedule, "axes": _prepare_axes,
         "cross": _prepare_cross}[case["op"]](case, seed)
    s["op"] = case["op"]
    return s


# ---------------------------------------------------------------------------- plain forms
def _plain_schedule(s):
    past, new, table = s["past"].long(), s["new"].long(), s["table"]
    bs, nb, t = s["block_size"], s["num_blocks"], s["tokens"]
    held = (past + bs - 1) // bs
    need = (past + new + bs - 1) // bs - held
    col = torch.arange(table.shape[1], device=DEV)
    mine = table[col[None, :] < held[:, None]].long()
    taken = torch.zeros(nb, dtype=torch.int64, device=DEV)
    taken[mine[(mine >= 0) & (mine < nb)]] = 1
    free = torch.nonzero(taken == 0)[:, 0]
    upto = torch.cumsum(need, 0)                       # blocks asked for up to each row
    ok = (need == 0) | (upto <= free.numel())
    given = torch.where(ok, new, torch.zeros_like(new))
    ok &= (given == 0) | (torch.cumsum(given, 0) <= t)   # rows past the token buffers
    given = torch.where(ok, given, torch.zeros_like(given))
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(given, 0)])
    need = torch.where(ok, need, torch.zeros_like(need))
    row = torch.repeat_interleave(torch.arange(past.numel(), device=DEV), need)
    nth = torch.arange(row.numel(), device=DEV) - (torch.cumsum(need, 0) - need)[row]
    table[row, held[row] + nth] = free[(upto - need)[row] + nth].int()
    i = torch.arange(t, device=DEV)
    of = torch.searchsorted(cu[1:], i, right=True).clamp(max=past.numel() - 1)
    live = i < cu[-1]
    pos = torch.where(live, past[of] + i - cu[of], torch.full_like(i, -1))
    block = table[of, pos.clamp(min=0) // bs].long()
    slot = torch.where(live & (block >= 0), block * bs + pos % bs, torch.full_like(i, -1))
    s["cu"].copy_(cu)
    s["slots"].copy_(slot)
    s["positions"].copy_(pos)
    s["total"].copy_(past + given)
    s["free"].copy_(free.numel() - need.sum())


def _plain_axes(s):
    hq, hkv, d, half = s["hq"], s["hkv"], s["d"], s["half"]
    if s["k"] is None:
        q, k, v = s["q"].split([hq * d, hkv * d, hkv * d], dim=1)
    else:
        q, k, v = s["q"], s["k"], s["v"]
    n = q.shape[0]
    at = s["pos"].long()[s["axis_dev"]].t()                      # [tokens, pairs]
    pair = torch.arange(half, device=DEV)
    c, w = s["cos"].float()[at, pair][:, None], s["sin"].float()[at, pair][:, None]

    def turned(x, heads):
        x = x.reshape(n, heads, d).float()
        if s["interleaved"]:
            a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
            r = torch.stack([a * c - b * w, b * c + a * w], -1).flatten(2)
        else:
            a, b = x[..., :half], x[..., half:2 * half]
            r = torch.cat([a * c - b * w, b * c + a * w], -1)
        return torch.cat([r, x[..., 2 * half:]], -1).to(s["q"].dtype)

    live = s["slots"] >= 0
    to = s["slots"][live].long()
    s["q_out"][live] = turned(q, hq).flatten(1)[live]
    s["kc"].view(-1, hkv, d)[to] = turned(k, hkv)[live]
    s["vc"].view(-1, hkv, d)[to] = v.reshape(n, hkv, d)[live]


def _plain_cross(s):
    hq, hkv, d, bs = s["hq"], s["hkv"], s["d"], s["bs"]
    g, b, mq, mk = hq // hkv, s["nk"].numel(), s["max_q"], s["max_k"]
    cu = s["cu"].long()
    i = torch.arange(s["q"].shape[0], device=DEV)
    of = torch.searchsorted(cu[1:], i, right=True)
    q = torch.zeros((b, mq, hq * d), dtype=torch.float32, device=DEV)
    q[of, i - cu[of]] = s["q"].float()
    q = q.view(b, mq, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * mq, d)
    j = torch.arange(mk, device=DEV)
    seen = j[None, :] < s["nk"][:, None]
    row = s["table"].long()[:, j // bs] * bs + j % bs
    row = torch.where(seen, row, torch.zeros_like(row))
    k = s["kc"].view(-1, hkv, d)[row].float().permute(0, 2, 3, 1)   # [b, hkv, d, mk]
    v = s["vc"].view(-1, hkv, d)[row].float().permute(0, 2, 1, 3)
    p = torch.matmul(q * (1.0 / math.sqrt(d)), k)
    p.masked_fill_(~seen[:, None, None, :], float("-inf"))
    top = p.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(b, hkv, g, mq, d).permute(0, 3, 1, 2, 4).reshape(b, mq, hq * d)
    lse = (top + torch.log(total)).view(b, hkv, g, mq).permute(0, 3, 1, 2).reshape(b, mq, hq)
    s["out"].copy_(o[of, i - cu[of]])
    s["lse"].copy_(lse[of, i - cu[of]])


# -------------------------------------------------------------------- the package's calls
def _own_schedule(s):
    from paged_kv_cache_231_gb300 import binding as B
    B.pkv_paged_schedule(s["past"], s["new"], s["table"], num_blocks=s["num_blocks"],
                         block_size=s["block_size"], num_tokens=s["tokens"],
                         cumulative_sequence_length=s["cu"], slot_mapping=s["slots"],
                         positions=s["positions"], total_seqlens=s["total"],
                         free_blocks=s["free"])


def _own_axes(s):
    from paged_kv_cache_231_gb300 import binding as B
    B.pkv_paged_append_rotary_axes(
        s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"], s["pos"],
        num_heads=s["hq"], kv_num_heads=s["hkv"], cos_cache=s["cos"], sin_cache=s["sin"],
        rotary_dim=2 * s["half"], pair_axis=s["axis"], rotary_interleaved=s["interleaved"],
        query_out=s["q_out"])


def _own_cross(s):
    from paged_kv_cache_231_gb300 import binding as B
    B.pkv_cross_attention(
        s["q"], s["kc"], s["vc"], s["cu"], s["nk"], s["table"], num_heads=s["hq"],
        kv_num_heads=s["hkv"], max_query_len=s["max_q"], output=s["out"], lse=s["lse"])


def run(s):
    if own:
        {"schedule": _own_schedule, "axes": _own_axes, "cross": _own_cross}[s["op"]](s)
    else:
        {"schedule": _plain_schedule, "axes": _plain_axes, "cross": _plain_cross}[s["op"]](s)
    names = {"schedule": ("cu", "slots", "positions", "total", "free", "table"),
             "axes": ("q_out", "kc", "vc"), "cross": ("out", "lse")}[s["op"]]
    return {n: s[n] for n in names}


# ------------------------------------------------------------------------------ definition
def _exact_schedule(s):
    past, new = s["past"].tolist(), s["new"].tolist()
    table, bs = s["table"].cpu().numpy().astype(np.int64), s["block_size"]
    held = [_ceil(p, bs) for p in past]
    taken = {int(x) for b, h in enumerate(held) for x in table[b, :h]}
    free = [x for x in range(s["num_blocks"]) if x not in taken]
    slots = np.full(s["tokens"], -1, np.int64)
    pos = np.full(s["tokens"], -1, np.int64)
    cu, total, at, used = [0], [], 0, 0
    for b, (p, n) in enumerate(zip(past, new)):
        need = _ceil(p + n, bs) - held[b]
        fits = (need == 0 or at + need <= len(free)) and cu[-1] + n <= s["tokens"]
        if fits:
            table[b, held[b]:held[b] + need] = free[at:at + need]
            used += need
            there = np.arange(p, p + n)
            pos[cu[-1]:cu[-1] + n] = there
            slots[cu[-1]:cu[-1] + n] = table[b, there // bs] * bs + there % bs
        at += need
        cu.append(cu[-1] + (n if fits else 0))
        total.append(p + (n if fits else 0))
    as32 = lambda x: torch.from_numpy(np.asarray(x, np.int32))  # noqa: E731
    return {"cu": as32(cu), "slots": as32(slots), "positions": as32(pos),
            "total": as32(total), "free": as32([len(free) - used]), "table": as32(table)}


def _exact_axes(s):
    hq, hkv, d, r = s["hq"], s["hkv"], s["d"], 2 * s["half"]
    x = s["q"] if s["k"] is None else torch.cat([s["q"], s["k"], s["v"]], 1)
    x = x.double().view(x.shape[0], hq + 2 * hkv, d).clone()
    of = torch.arange(r, device=DEV)
    pair = of // 2 if s["interleaved"] else of % s["half"]
    first = of % 2 == 0 if s["interleaved"] else of < s["half"]
    other = of ^ 1 if s["interleaved"] else (of + s["half"]) % r
    where = s["pos"].long()[s["axis_dev"][pair]].t()
    turn = s["cos"].double()[where, pair] + 1j * s["sin"].double()[where, pair]
    own_part, partner = x[:, :hq + hkv, :r], x[:, :hq + hkv, other]
    sign = torch.where(first, -1.0, 1.0).double()
    x[:, :hq + hkv, :r] = own_part * turn.real[:, None] + sign * partner * turn.imag[:, None]
    q_out, kc, vc = s["q_out"].double(), s["kc"].double(), s["vc"].double()
    live = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"][live].long()
    q_out[live] = x[live, :hq].flatten(1)
    kc.view(-1, hkv, d)[at] = x[live, hq:hq + hkv]
    vc.view(-1, hkv, d)[at] = x[live, hq + hkv:]
    return {"q_out": q_out, "kc": kc, "vc": vc}


def _exact_cross(s):
    hq, hkv, d, bs = s["hq"], s["hkv"], s["d"], s["bs"]
    cu, nk = s["cu"].tolist(), s["nk"].tolist()
    out = torch.zeros((cu[-1], hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((cu[-1], hq), float("-inf"), dtype=torch.float64, device=DEV)
    for b, n in enumerate(nk):
        if n == 0:
            continue
        blocks = s["table"][b, :_ceil(n, bs)].long()
        k = s["kc"][blocks].flatten(0, 1)[:n].double().repeat_interleave(hq // hkv, 1)
        v = s["vc"][blocks].flatten(0, 1)[:n].double().repeat_interleave(hq // hkv, 1)
        q = s["q"][cu[b]:cu[b + 1]].double().view(-1, hq, d)
        score = torch.einsum("thd,nhd->htn", q, k) / math.sqrt(d)
        lse[cu[b]:cu[b + 1]] = torch.logsumexp(score, -1).t()
        out[cu[b]:cu[b + 1]] = torch.einsum("htn,nhd->thd", torch.softmax(score, -1), v)
    return {"out": out.flatten(1), "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"schedule": _exact_schedule, "axes": _exact_axes,
            "cross": _exact_cross}[case["op"]](s)
