"""GPU parity of pkv_paged_schedule: whole numbers, equal to the oracle's."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as orc
from paged_kv_cache_231_gb300 import binding as B

from .step_util import DEV, i32, paged_pool

pytestmark = pytest.mark.gpu
NAMES = ("cu", "slots", "positions", "total", "free", "table")


def run(past, new, table, *, status=True, **kw):
    t, st = i32(table), torch.zeros(1, dtype=torch.int32, device=DEV)
    got = B.pkv_paged_schedule(i32(past), i32(new), t, device_status=st if status else None, **kw)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in got] + [t.cpu().numpy()], int(st.item())


def check(past, new, table, **kw):
    got, status = run(past, new, table, **kw)
    *ref, rstatus = orc.schedule(past, new, table, **kw)
    for name, g, r in zip(NAMES, got, ref):
        np.testing.assert_array_equal(g.reshape(-1), np.asarray(r).reshape(-1), err_msg=name)
    assert status == rstatus
    return got


def drawn(seed, rows, past, new, block_size, *, spare=0, idle=0.2):
    rng = np.random.default_rng(seed)
    p = rng.integers(0, past + 1, rows)
    n = rng.integers(1, new + 1, rows) * (rng.random(rows) > idle)
    asked = int(sum(-(-(a + b) // block_size) + -a // block_size for a, b in zip(p, n)))
    table, blocks = paged_pool(rng, p, block_size, -(-(past + new) // block_size) + 1,
                               max(asked + spare, 1 - int(p.sum() > 0)))
    return p, n, table, max(blocks, 1)


@pytest.mark.parametrize("rows,past,new,bs", [
    (1, 0, 1, 16), (1, 5, 1, 1), (2, 40, 1, 16), (3, 100, 70, 8), (64, 900, 1, 16),
    (64, 300, 5, 7), (33, 0, 257, 24), (1000, 60, 9, 4), (1025, 70, 3, 16), (2049, 33, 40, 8),
    (7, 5000, 3000, 1), (5, 20000, 9000, 16)])
def test_matches_oracle(rows, past, new, bs):
    p, n, table, blocks = drawn(rows * 7 + bs, rows, past, new, bs, spare=5)
    tokens = int(n.sum())
    for t in (tokens, tokens + 37):
        check(p, n, table, num_blocks=blocks, block_size=bs, num_tokens=t)


@pytest.mark.parametrize("short", [1, 2, 9, 40])
@pytest.mark.parametrize("seed", [1, 2])
def test_pool_too_small(seed, short):
    p, n, table, blocks = drawn(seed, 70, 100, 50, 8, spare=-short)
    got = check(p, n, table, num_blocks=blocks, block_size=8, num_tokens=int(n.sum()))
    assert got[0][-1] < n.sum()


@pytest.mark.parametrize("cut", [1, 10, 400])
def test_token_buffers_too_small(cut):
    p, n, table, blocks = drawn(5, 90, 100, 30, 16, spare=3)
    check(p, n, table, num_blocks=blocks, block_size=16, num_tokens=max(0, int(n.sum()) - cut))


def test_no_tokens_at_all():
    p, n, table, blocks = drawn(6, 20, 100, 30, 16, spare=3)
    got = check(p, 0 * n, table, num_blocks=blocks, block_size=16, num_tokens=0)
    assert not got[0].any()


def test_invalid_lengths_and_table_rows():
    past, new = [-3, 5, 40, 7, 2**31 - 1, 6, 0], [4, -1, 30, 2, 1, 2**31 - 1, 3]
    table = np.full((7, 4), -1, np.int32)          # limit 4 * 16 = 64 tokens
    table[1, 0], table[2, :3], table[3, 0], table[5, 0] = 9, [3, 77, 11], -8, 2
    got = check(past, new, table, num_blocks=20, block_size=16, num_tokens=50)
    assert got[0].tolist() == [0, 0, 0, 0, 2, 2, 2, 5]   # row 3: its block is missing
    assert got[1].tolist()[:2] == [-1, -1]


def test_holes_and_shared_blocks():
    # rows 0 and 1 share their first blocks; row 2's first block was given up
    table = np.array([[4, 6, 1, -1], [4, 6, 3, -1], [-1, 0, -1, -1]], np.int32)
    got = check([20, 21, 13], [9, 1, 5], table, num_blocks=9, block_size=8, num_tokens=20)
    assert got[5].tolist() == [[4, 6, 1, 2], [4, 6, 3, -1], [-1, 0, 5, -1]]


def test_large_pool_and_many_groups():
    # free blocks far apart: all but every 997th of 1 048 576 blocks are held
    blocks = 1 << 20
    held = np.array([x for x in range(blocks) if x % 997], np.int32)
    rows, mb = 8, (len(held) + 7) // 8 + 200
    table, past = np.full((rows, mb), -1, np.int32), []
    for b, part in enumerate(np.array_split(held, rows)):
        table[b, :len(part)] = part
        past.append(len(part))
    got, status = run(past, [100] * rows, table, num_blocks=blocks, block_size=1,
                      num_tokens=800)
    free = [x for x in range(blocks) if x % 997 == 0]
    assert status == 0 and got[1].tolist() == free[:800]
    assert got[4].tolist() == [len(free) - 800]


def test_result_depends_on_the_inputs_alone():
    # a second call on the table the first one wrote gives the same, bit for bit
    p, n, table, blocks = drawn(9, 300, 200, 40, 16, spare=11)
    kw = dict(num_blocks=blocks, block_size=16, num_tokens=int(n.sum()))
    a, _ = run(p, n, table, **kw)
    b, _ = run(p, n, a[5], status=False, **kw)
    for x, y in zip(a, b):
        np.testing.assert_array_equal(x, y)


def test_unaligned_outputs_and_unwritten_entries():
    p, n, table, blocks = drawn(10, 50, 100, 40, 8, spare=2)
    T = int(n.sum())
    buf = torch.full((3, T + 8), -77, dtype=torch.int32, device=DEV)
    st = i32(table)
    B.pkv_paged_schedule(i32(p), i32(n), st, num_blocks=blocks, block_size=8, num_tokens=T,
                         slot_mapping=buf[0, 1:T + 1], positions=buf[1, 3:T + 3])
    ref = orc.schedule(p, n, table, num_blocks=blocks, block_size=8, num_tokens=T)
    np.testing.assert_array_equal(buf[0, 1:T + 1].cpu().numpy(), ref[1])
    np.testing.assert_array_equal(buf[1, 3:T + 3].cpu().numpy(), ref[2])
    assert (buf[0, [0, -1]] == -77).all() and (buf[1, :3] == -77).all()
    assert (buf[1, T + 3:] == -77).all() and (buf[2] == -77).all()


def test_captured_and_replayed_on_a_side_stream():
    p, n, table, blocks = drawn(11, 64, 200, 1, 16, spare=90, idle=0.0)
    past, new, t = i32(p), i32(n), i32(table)
    kw = dict(num_blocks=blocks, block_size=16, num_tokens=80)
    out = B.pkv_paged_schedule(past, new, t, **kw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        B.pkv_paged_schedule(past, new, t, cumulative_sequence_length=out[0],
                             slot_mapping=out[1], positions=out[2], total_seqlens=out[3],
                             free_blocks=out[4], **kw)
        past.copy_(out[3])            # the next step goes on where this one ended
    ref_table, ref_past = table, p
    for step in range(40):
        g.replay()
        torch.cuda.synchronize()
        *ref, status = orc.schedule(ref_past, n, ref_table, **kw)
        ref_table, ref_past = ref[5], ref[3]
        # late in the run the pool is empty and rows reach the end of the table
        assert not status & ~(orc.NO_BLOCKS | orc.BAD_BLOCK)
        for name, x, r in zip(NAMES, [*out, t], ref):
            np.testing.assert_array_equal(x.cpu().numpy().reshape(-1),
                                          np.asarray(r).reshape(-1), err_msg=f"{name} {step}")


@pytest.mark.parametrize("rows,past,new,bs,cut", [
    (150, 3000, 1200, 16, -5), (150, 3000, 1200, 24, 900), (40, 500, 5000, 1, 0),
    (8192, 40, 40, 8, -1), (1, 3, 90000, 32, -30000)])
def test_very_many_tokens(rows, past, new, bs, cut):
    # so many that their slots are a kernel of their own; a hole among the held blocks
    p, n, table, blocks = drawn(rows + bs, rows, past, new, bs, spare=4, idle=0.1)
    if p[0] % bs:
        table[0, p[0] // bs] = -1
    tokens = int(n.sum()) - cut
    assert tokens >= 65536
    kw = dict(num_blocks=blocks, block_size=bs, num_tokens=tokens)
    got = check(p, n, table, **kw)
    buf = torch.full((2, tokens + 9), 5, dtype=torch.int32, device=DEV)   # not 16-byte aligned
    slots, pos = buf[0, 1:tokens + 1], buf[1, 3:tokens + 3]
    more, _ = run(p, n, table, slot_mapping=slots, positions=pos, **kw)
    for x, y in zip(got, more):
        np.testing.assert_array_equal(x, y)
    assert buf[0, 0] == 5 and (buf[0, tokens + 1:] == 5).all()
    assert (buf[1, :3] == 5).all() and (buf[1, tokens + 3:] == 5).all()


def test_very_many_tokens_in_a_graph():
    p, n, table, blocks = drawn(3, 200, 3000, 900, 16, spare=4, idle=0.1)
    kw = dict(num_blocks=blocks, block_size=16, num_tokens=int(n.sum()))
    want, _ = run(p, n, table, **kw)
    past, new, t = i32(p), i32(n), i32(table)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = B.pkv_paged_schedule(past, new, t, **kw)
    for _ in range(3):
        t.copy_(i32(table))
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(list(out) + [t], want):
            np.testing.assert_array_equal(x.cpu().numpy(), y)
