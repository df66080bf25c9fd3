"""GPU parity of pkv_paged_append_norm_rotary."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as orc
from paged_kv_cache_231_gb300 import binding as B

from .step_util import DEV, TYPES, half_step, i32, wide
from .test_gpu_append_axes import Case as Axes

pytestmark = pytest.mark.gpu


class Case(Axes):
    def __init__(self, seed, tokens, *, weight="f32", weights="qk", epsilon=1e-5, spread=1.0, **kw):
        super().__init__(seed, tokens, **kw)
        gen = torch.Generator()
        gen.manual_seed(seed + 1)
        wt = TYPES[weight]
        new = lambda: (1 + 0.3 * torch.randn(self.d, generator=gen)).to(wt)  # noqa: E731
        self.qw, self.kw = (new() if x in weights else None for x in "qk")
        self.eps = epsilon
        for x in (self.q, self.k, self.v):
            if x is not None:
                x *= spread

    def call(self, q, k, v, kc, vc, slots, pos, out, **kw):
        up = lambda x: None if x is None else x.to(DEV)  # noqa: E731
        return B.pkv_paged_append_norm_rotary(
            q, k, v, kc, vc, slots, pos, num_heads=self.hq, kv_num_heads=self.hkv,
            query_weight=up(self.qw), key_weight=up(self.kw), epsilon=self.eps,
            cos_cache=up(self.cos) if self.r else None, sin_cache=up(self.sin) if self.r else None,
            rotary_dim=self.r, pair_axis=self.axis, rotary_interleaved=self.interleaved,
            query_out=out, **kw)

    def check(self, status=0):
        kc, vc = self.kc.to(DEV), self.vc.to(DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        up = lambda x: None if x is None else x.to(DEV)  # noqa: E731
        out = torch.full((self.T, self.hq * self.d), 7.0, dtype=self.t, device=DEV) \
            if self.query else None
        got = self.call(up(self.q), up(self.k), up(self.v), kc, vc, i32(self.slots),
                        i32(self.pos) if self.r else None, out, device_status=st)
        assert got is out
        torch.cuda.synchronize()
        if self.packed:
            x = wide(self.q).reshape(self.T, -1, self.d)
            q, k, v = np.split(x, [self.hq, self.hq + self.hkv], axis=1)
        else:
            k, v = (wide(x).reshape(self.T, -1, self.d) for x in (self.k, self.v))
            q = wide(self.q).reshape(self.T, -1, self.d) if self.query else None
        pool = (-1, self.hkv, self.d)
        w = lambda x: None if x is None else wide(x)  # noqa: E731
        start = np.full((self.T, self.hq, self.d), 7.0)
        rq, rk, rv, sq, sk, rst = orc.append_norm(
            q, k, v, wide(self.kc).reshape(pool), wide(self.vc).reshape(pool), self.slots, self.pos,
            wide(self.cos), wide(self.sin), num_heads=self.hq, kv_num_heads=self.hkv,
            rotary_dim=self.r, pair_axis=self.axis, interleaved=self.interleaved,
            q_out=start if self.query else None, query_weight=w(self.qw), key_weight=w(self.kw),
            epsilon=self.eps)
        assert int(st.item()) == rst == status
        # 32 bits: a sum of D <= 256 squares errs by at most 2^-19 of itself in this order or any
        # tree, its root by half of that, the reciprocal root by 2^-22, three products by 2^-24
        # each: 2^-19 in all; the turn's two products and sum by 2^-22 of their magnitudes. Then
        # one rounding, which is 2^-25 absolute below fp16's normal numbers.
        tiny = 2.0 ** -25 * 1.01 if self.t == torch.float16 else 1e-38
        for g, ref, size in ((out, rq, sq), (kc, rk, sk)):
            if g is None:
                continue
            err = np.abs(wide(g).reshape(ref.shape) - ref)
            tol = (half_step(self.t) * 1.01 + 2.0 ** -18) * np.abs(ref) + 2.0 ** -18 * size + tiny
            assert (err <= tol).all(), (float(err.max()), np.argwhere(~(err <= tol))[:4].tolist())
        assert np.array_equal(wide(vc).reshape(rv.shape), rv)
        # what no token is written to stays as it was, bit for bit
        mine = np.zeros(kc.shape[0] * kc.shape[1], bool)
        mine[self.slots[(self.slots >= 0) & (self.slots < len(mine))]] = True
        rest = torch.from_numpy(~mine)
        assert torch.equal(kc.cpu().reshape(pool)[rest], self.kc.reshape(pool)[rest])
        return out, kc, vc


@pytest.mark.parametrize("head_size,rotary_dim", [(64, 64), (64, 32), (128, 128), (128, 64),
                                                  (128, 16), (256, 256), (256, 128), (96, 96),
                                                  (80, 40), (8, 8), (128, 20), (64, 0), (128, 2),
                                                  (248, 248)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_sizes(head_size, rotary_dim, interleaved):
    Case(1, 37, head_size=head_size, rotary_dim=rotary_dim, interleaved=interleaved,
         axes=1 if rotary_dim else 0).check()


@pytest.mark.parametrize("tokens", [1, 2, 3, 30, 700, 2000])
@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (12, 4), (32, 8), (40, 8), (64, 8), (128, 2)])
def test_tokens_and_heads(tokens, heads, kv):
    if tokens * heads > 30000:
        tokens = 30000 // heads
    Case(2, tokens, num_heads=heads, kv_heads=kv, head_size=128, rotary_dim=128, axes=1,
         packed=True, dtype="bf16", weight="bf16").check()


@pytest.mark.parametrize("dtype,table,weight", [("f16", "f16", "f16"), ("f16", "f32", "f32"),
                                                ("bf16", "bf16", "f32"), ("bf16", "f32", "bf16")])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("axes,turns", [(1, False), (3, True), (8, False)])
def test_types_and_axes(dtype, table, weight, packed, axes, turns):
    Case(3, 61, dtype=dtype, table=table, weight=weight, packed=packed, axes=axes, turns=turns,
         pad=(0, 7, 60)).check()


@pytest.mark.parametrize("tokens,heads,kv,head_size,rotary_dim,interleaved", [
    # one, two and four tokens a thread, a block for each group or blocks that stay
    (200, 16, 4, 256, 256, False), (500, 16, 4, 256, 256, True), (900, 16, 4, 256, 64, False),
    (1300, 16, 4, 256, 256, False), (1500, 4, 2, 256, 64, True), (3000, 4, 2, 256, 32, False),
    (4000, 4, 2, 256, 64, True), (5000, 1, 1, 64, 32, False), (9000, 6, 3, 128, 16, True),
    (30000, 2, 1, 64, 16, False)])
def test_tokens_of_a_thread(tokens, heads, kv, head_size, rotary_dim, interleaved):
    Case(10, tokens, num_heads=heads, kv_heads=kv, head_size=head_size, rotary_dim=rotary_dim,
         interleaved=interleaved, axes=2, pad=(1, tokens - 1)).check()


@pytest.mark.parametrize("tokens", [40, 2000])
def test_packed_rows_whose_queries_are_left(tokens):
    c = Case(11, tokens, packed=True, head_size=128, rotary_dim=64, axes=1)
    kc, vc = (x.to(DEV) for x in (c.kc, c.vc))
    want = [x.cpu() for x in c.check()]
    args = dict(num_heads=c.hq, kv_num_heads=c.hkv, key_weight=c.kw.to(DEV), epsilon=c.eps,
                query_weight=c.qw.to(DEV), cos_cache=c.cos.to(DEV), sin_cache=c.sin.to(DEV),
                rotary_dim=c.r, pair_axis=c.axis)
    assert B.pkv_paged_append_norm_rotary(c.q.to(DEV), None, None, kc, vc, i32(c.slots),
                                          i32(c.pos), rotate_query=False, **args) is None
    torch.cuda.synchronize()
    assert torch.equal(kc.cpu(), want[1]) and torch.equal(vc.cpu(), want[2])


@pytest.mark.parametrize("weights", ["q", "k", "qk"])
@pytest.mark.parametrize("head_size", [128, 72])
def test_one_side_alone(weights, head_size):
    Case(4, 20, head_size=head_size, rotary_dim=head_size, weights=weights).check()


@pytest.mark.parametrize("head_size", [64, 72])
def test_without_queries(head_size):
    Case(5, 40, query=False, head_size=head_size, rotary_dim=32).check()


@pytest.mark.parametrize("head_size", [128, 40])
@pytest.mark.parametrize("dtype,spread", [("f16", 1e-3), ("f16", 1e3), ("bf16", 1e12),
                                          ("bf16", 1e-12), ("f16", 0.0)])
def test_magnitudes(head_size, dtype, spread):
    Case(6, 30, head_size=head_size, rotary_dim=head_size, axes=1, dtype=dtype,
         spread=spread).check()


@pytest.mark.parametrize("head_size", [64, 72])
@pytest.mark.parametrize("tokens", [50, 2100])
def test_bad_slots_and_positions(head_size, tokens):
    c = Case(7, tokens, head_size=head_size, rotary_dim=64, axes=2, pad=(3,))
    c.slots[5] = c.nb * c.bs
    c.slots[6] = 2 ** 31 - 1
    c.check(status=B.DEV_BAD_SLOT)
    c.pos[1, 8], c.pos[0, 9] = 300, -1
    c.check(status=B.DEV_BAD_SLOT | B.DEV_BAD_POSITION)


def test_a_row_that_is_not_finite_stays_alone():
    c = Case(8, 30, head_size=128, rotary_dim=128, axes=1)
    want = [x.cpu() for x in c.check()]
    c.q[4, :128] = float("nan")
    c.k[9, 5] = float("inf")
    out = torch.zeros((30, c.hq * c.d), dtype=c.t, device=DEV)
    kc, vc = c.kc.to(DEV), c.vc.to(DEV)
    c.call(c.q.to(DEV), c.k.to(DEV), c.v.to(DEV), kc, vc, i32(c.slots), i32(c.pos), out)
    torch.cuda.synchronize()
    got = out.cpu()
    assert torch.isnan(got[4, :128]).all()
    got[4, :128] = want[0][4, :128]
    assert torch.equal(got, want[0])
    pool = (-1, c.hkv, c.d)
    keys, ref = kc.cpu().reshape(pool), want[1].reshape(pool)
    assert torch.isnan(keys[c.slots[9], 0]).any()
    keys[c.slots[9], 0] = ref[c.slots[9], 0]
    assert torch.equal(keys, ref)


def test_graph_and_stream():
    c = Case(9, 900, num_heads=32, kv_heads=8, head_size=128, rotary_dim=128, axes=1)
    want = [x.cpu() for x in c.check()]
    args = [c.q.to(DEV), c.k.to(DEV), c.v.to(DEV), c.kc.to(DEV), c.vc.to(DEV), i32(c.slots),
            i32(c.pos)]
    out = torch.full((900, c.hq * c.d), 7.0, dtype=c.t, device=DEV)
    qw, kw, cos, sin = (x.to(DEV) for x in (c.qw, c.kw, c.cos, c.sin))
    call = lambda **more: B.pkv_paged_append_norm_rotary(  # noqa: E731
        *args, num_heads=c.hq, kv_num_heads=c.hkv, query_weight=qw, key_weight=kw, epsilon=c.eps,
        cos_cache=cos, sin_cache=sin, rotary_dim=c.r, pair_axis=c.axis, **more)
    call(query_out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(query_out=out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want[0]) and torch.equal(args[3].cpu(), want[1])
    s = torch.cuda.Stream()
    other = call(stream=s)
    s.synchronize()
    assert torch.equal(other.cpu(), want[0])
