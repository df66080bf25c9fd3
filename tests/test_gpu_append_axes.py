"""GPU parity of pkv_paged_append_rotary_axes."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as orc
from paged_kv_cache_231_gb300 import binding as B

from .step_util import DEV, TYPES, half_step, i32, wide

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, seed, tokens, *, num_heads=4, kv_heads=2, head_size=64, rotary_dim=64,
                 axes=3, dtype="f16", table="f32", packed=False, interleaved=False,
                 block_size=16, positions=300, pad=(), turns=False, query=True):
        rng = np.random.default_rng(seed)
        gen = torch.Generator()
        gen.manual_seed(seed)
        self.t, self.tt = TYPES[dtype], TYPES[table]
        self.T, self.hq, self.hkv, self.d = tokens, num_heads, kv_heads, head_size
        self.r, self.half, self.axes = rotary_dim, rotary_dim // 2, axes
        new = lambda *s: torch.randn(s, generator=gen).to(self.t)  # noqa: E731
        hidden = (num_heads + 2 * kv_heads) * head_size
        self.packed, self.query = packed, query or packed
        if packed:
            self.q, self.k, self.v = new(tokens, hidden), None, None
        else:
            self.q = new(tokens, num_heads * head_size) if query else None
            self.k, self.v = (new(tokens, kv_heads * head_size) for _ in range(2))
        self.nb, self.bs = -(-tokens // block_size) + 2, block_size
        self.slots = rng.permutation(self.nb * block_size)[:tokens].astype(np.int32)
        for i in pad:
            self.slots[i] = -1 - i
        self.pos = rng.integers(0, positions, (axes, tokens)).astype(np.int32)
        for i in pad:   # nothing of a padding token is looked at
            self.pos[:, i] = -(2 ** 31)
        ang = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(self.half) / max(1, self.half))
        self.cos, self.sin = (torch.from_numpy(f(ang)).to(self.tt) for f in (np.cos, np.sin))
        n = [self.half // axes + (a < self.half % axes) for a in range(axes)] if axes else []
        self.axis = B.rotary_pair_axis(n, by_turns=turns) if axes else []
        self.interleaved = interleaved
        self.kc, self.vc = (new(self.nb, block_size, kv_heads, head_size) for _ in range(2))

    def gpu(self, **kw):
        kc, vc = self.kc.to(DEV), self.vc.to(DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        up = lambda x: None if x is None else x.to(DEV)  # noqa: E731
        out = None
        if self.query:
            out = torch.full((self.T, self.hq * self.d), 7.0, dtype=self.t, device=DEV)
        got = B.pkv_paged_append_rotary_axes(
            up(self.q), up(self.k), up(self.v), kc, vc, i32(self.slots),
            i32(self.pos) if self.r else None, num_heads=self.hq, kv_num_heads=self.hkv,
            cos_cache=up(self.cos) if self.r else None, sin_cache=up(self.sin) if self.r else None,
            rotary_dim=self.r, pair_axis=self.axis, rotary_interleaved=self.interleaved,
            query_out=out, device_status=st, **kw)
        assert got is out
        torch.cuda.synchronize()
        return out, kc, vc, int(st.item())

    def check(self, **kw):
        out, kc, vc, status = self.gpu(**kw)
        d = self.d
        rows = [self.q, self.k, self.v]
        if self.packed:
            rows = self.q.split([self.hq * d, self.hkv * d, self.hkv * d], 1)
        q, k, v = (None if x is None else wide(x).reshape(self.T, -1, d) for x in rows)
        pool = lambda x: wide(x).reshape(-1, self.hkv, d)  # noqa: E731
        q_out = np.full((self.T, self.hq, d), 7.0) if self.query else None
        rq, rk, rv, slack_q, slack_k, rstatus = orc.append_axes(
            q, k, v, pool(self.kc), pool(self.vc), self.slots, self.pos, wide(self.cos),
            wide(self.sin), num_heads=self.hq, kv_num_heads=self.hkv, rotary_dim=self.r,
            pair_axis=self.axis, interleaved=self.interleaved, q_out=q_out)
        assert status == rstatus
        np.testing.assert_array_equal(pool(vc), rv)
        for name, got, ref, slack in (("key", kc, rk, slack_k), ("query", out, rq, slack_q)):
            if ref is None:
                continue
            # two products and a sum in fp32 (each off by 2^-24 of its size), then one rounding
            # to the type; below fp16's normal range a step is 2^-24
            tol = np.where(slack > 0, half_step(self.t) * np.abs(ref) + 3 * 2.0 ** -24 * slack, 0)
            tol = np.where(slack > 0, np.maximum(tol, 2.0 ** -25) * 1.001, 0)
            err = np.abs(wide(got).reshape(ref.shape) - ref)
            assert (err <= tol).all(), (name, float((err - tol).max()))


@pytest.mark.parametrize("dtype,table", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"),
                                         ("bf16", "f32")])
@pytest.mark.parametrize("kw", [
    dict(tokens=1), dict(tokens=37, packed=True), dict(tokens=5, interleaved=True),
    dict(tokens=19, head_size=128, rotary_dim=128, num_heads=8, kv_heads=2, packed=True),
    dict(tokens=9, head_size=128, rotary_dim=64, turns=True),
    dict(tokens=9, head_size=128, rotary_dim=96, interleaved=True, axes=2),
    dict(tokens=8, head_size=128, rotary_dim=20, axes=4),       # pairs across chunks
    dict(tokens=8, head_size=72, rotary_dim=6, interleaved=True, axes=1),
    dict(tokens=6, head_size=256, rotary_dim=256, num_heads=3, kv_heads=1, axes=8),
    dict(tokens=4, head_size=80, rotary_dim=80, num_heads=5, kv_heads=5),
    dict(tokens=70, num_heads=40, kv_heads=8, head_size=64, rotary_dim=32, packed=True),
    dict(tokens=12, rotary_dim=0, axes=0), dict(tokens=12, rotary_dim=0, axes=0, query=False),
    dict(tokens=33, query=False, block_size=7), dict(tokens=21, pad=(0, 3, 4, 20)),
], ids=str)
def test_matches_oracle(kw, dtype, table):
    Case(3, dtype=dtype, table=table, **kw).check()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_bad_positions_and_slots(packed, interleaved):
    c = Case(4, 12, packed=packed, interleaved=interleaved, pad=(5,))
    c.pos[0, 2], c.pos[1, 3], c.pos[2, 4] = -1, 300, 2 ** 31 - 1
    c.slots[7], c.slots[8], c.slots[2] = c.nb * c.bs, 2 ** 31 - 1, c.nb * c.bs + 5
    c.check()


def test_position_of_an_axis_that_no_pair_uses():
    c = Case(5, 6, axes=3)
    c.axis = [0 if a == 1 else a for a in c.axis]
    c.pos[1] = -9
    c.check()


def test_every_token_is_padding():
    c = Case(6, 4, pad=(0, 1, 2, 3))
    out, kc, vc, status = c.gpu()
    assert status == 0 and (out == 7).all()
    assert torch.equal(kc.cpu(), c.kc) and torch.equal(vc.cpu(), c.vc)


def test_no_tokens():
    c = Case(6, 0)
    assert c.gpu()[3] == 0


def test_equals_the_one_axis_append_in_paged_attention():
    # with one axis the pool gets what the paged scatter with rotary writes, bit for bit
    c = Case(7, 40, axes=1, table="f16", head_size=128, rotary_dim=128)
    past, bt = 23, np.random.default_rng(1).permutation(c.nb)[:4].astype(np.int32)
    c.pos = (past + np.arange(40, dtype=np.int32))[None]
    at = past + np.arange(40)
    c.slots = (bt[at // c.bs] * c.bs + at % c.bs).astype(np.int32)
    _, kc, vc, _ = c.gpu()
    kc2, vc2 = c.kc.to(DEV), c.vc.to(DEV)
    B.pkv_paged_scatter_kv(c.q.to(DEV), c.k.to(DEV), c.v.to(DEV), kc2, vc2, i32([0, 40]),
                           i32([past]), i32(bt[None]), num_heads=c.hq, kv_num_heads=c.hkv,
                           cos_cache=c.cos.to(DEV), sin_cache=c.sin.to(DEV), rotary_dim=128)
    torch.cuda.synchronize()
    assert torch.equal(vc, vc2)
    c.check()
    step = (kc.float() - kc2.float()).abs() <= 2 * half_step(c.t) * kc.float().abs() + 2.0 ** -24
    assert step.all()


def test_captured_and_replayed():
    c = Case(8, 30, packed=True)
    ref = c.gpu()
    kc, vc, q = c.kc.to(DEV), c.vc.to(DEV), c.q.to(DEV)
    slots, pos, cos, sin = i32(c.slots), i32(c.pos), c.cos.to(DEV), c.sin.to(DEV)
    out = torch.full_like(ref[0], 7.0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.pkv_paged_append_rotary_axes(q, None, None, kc, vc, slots, pos, num_heads=c.hq,
                                       kv_num_heads=c.hkv, cos_cache=cos, sin_cache=sin,
                                       rotary_dim=c.r, pair_axis=c.axis, query_out=out)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref[0]) and torch.equal(kc, ref[1]) and torch.equal(vc, ref[2])


def _slices_give_the_whole(c, step):
    """One call over all tokens equals calls over `step` of them at a time, bit for bit."""
    whole = c.gpu()
    kc, vc = c.kc.to(DEV), c.vc.to(DEV)
    out = torch.full_like(whole[0], 7.0) if c.query else None
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    cos, sin = c.cos.to(DEV), c.sin.to(DEV)
    for t in range(0, c.T, step):
        part = lambda x: None if x is None else x[t:t + step].contiguous().to(DEV)  # noqa: E731
        B.pkv_paged_append_rotary_axes(
            part(c.q), part(c.k), part(c.v), kc, vc, i32(c.slots[t:t + step]),
            i32(c.pos[:, t:t + step]), num_heads=c.hq, kv_num_heads=c.hkv, cos_cache=cos,
            sin_cache=sin, rotary_dim=c.r, pair_axis=c.axis, rotary_interleaved=c.interleaved,
            query_out=None if out is None else out[t:t + step], rotate_query=out is not None,
            device_status=st)
    torch.cuda.synchronize()
    if out is not None:
        assert torch.equal(out, whole[0])
    assert torch.equal(kc, whole[1]) and torch.equal(vc, whole[2])
    assert int(st.item()) == whole[3]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kw", [
    dict(tokens=2433, num_heads=16, kv_heads=4, head_size=128, rotary_dim=128),
    dict(tokens=1500, num_heads=16, kv_heads=4, head_size=128, rotary_dim=64, packed=True),
    dict(tokens=1217, num_heads=9, kv_heads=9, head_size=128, rotary_dim=0, axes=0, query=False),
    dict(tokens=10001, num_heads=4, kv_heads=2, head_size=64, rotary_dim=64, turns=True),
    dict(tokens=30007, num_heads=1, kv_heads=1, head_size=64, rotary_dim=32),
    dict(tokens=1300, num_heads=96, kv_heads=8, head_size=128, rotary_dim=128, axes=2),
], ids=str)
def test_many_tokens_equal_few_at_a_time(kw, interleaved):
    c = Case(9, interleaved=interleaved, pad=(1, 2, 700, kw["tokens"] - 1), **kw)
    if c.r:
        c.pos[0, 5], c.pos[-1, 900] = -4, 300
    c.slots[44] = c.nb * c.bs
    if c.r == 0:
        c.pos = np.zeros((1, c.T), np.int32)
    _slices_give_the_whole(c, 500)


def test_many_tokens_match_the_oracle():
    c = Case(10, 1290, num_heads=16, kv_heads=4, head_size=128, rotary_dim=128, dtype="bf16",
             packed=True, turns=True, pad=(0, 77, 1289))
    c.pos[1, 1000] = 300
    c.check()


@pytest.mark.parametrize("kw", [
    dict(tokens=320000, head_size=8, rotary_dim=0, axes=0),
    dict(tokens=100001, head_size=16, rotary_dim=16, axes=2),
    dict(tokens=160001, head_size=16, rotary_dim=16, axes=2),
    dict(tokens=160001, head_size=16, rotary_dim=16, axes=2, interleaved=True),
], ids=str)
def test_many_tokens_of_tiny_heads(kw):
    # a block holds more tokens than threads
    Case(12, num_heads=1, kv_heads=1, query=False, pad=(0, 999, 1500), **kw).check()


def test_pool_rows_past_32_bit_offsets():
    c = Case(11, 40, num_heads=8, kv_heads=8, head_size=128, rotary_dim=128)
    want = c.gpu()
    first = 2 ** 31 // (c.bs * 8 * 128) + 3
    kc = torch.zeros((first + c.nb, c.bs, 8, 128), dtype=c.t, device=DEV)
    vc = torch.zeros_like(kc)
    kc[first:], vc[first:] = c.kc.to(DEV), c.vc.to(DEV)
    out = B.pkv_paged_append_rotary_axes(
        c.q.to(DEV), c.k.to(DEV), c.v.to(DEV), kc, vc, i32(c.slots + first * c.bs), i32(c.pos),
        num_heads=8, kv_num_heads=8, cos_cache=c.cos.to(DEV), sin_cache=c.sin.to(DEV),
        rotary_dim=128, pair_axis=c.axis)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])
    assert torch.equal(kc[first:], want[1]) and torch.equal(vc[first:], want[2])
