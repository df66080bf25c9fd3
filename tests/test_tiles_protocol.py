"""The order in which the roles of the cross attention's kernel for many rows touch shared memory,
as a graph of what waits for what (no GPU). Two loaders, two issuers of products and two halves of
four softmax warps go through the same parts; a ring holds the key masks of a few steps, another
the K and V tiles. Every write that takes the place of older data must stand behind all reads of
it by way of the waits."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "paged_kv_cache_231_gb300", "csrc", "cross_tiles.cu")


def constants():
    with open(SOURCE) as f:
        text = f.read()
    wide, narrow = map(int, re.search(r"kStages = D == 128 \? (\d+) : (\d+)", text).groups())
    masks = int(re.search(r"constexpr int kMasks = (\d+);", text).group(1))
    # what the loader of keys waits for in front of new masks, with an even number of stages
    assert re.search(r"!kAlternate && kv == 0 && use >= 2u \* kMasks &&\s+"
                     r"!other_found\(use \+ 2 \+ L::kStages - 2 \* kMasks\)", text)
    return {128: wide, 64: narrow}, masks


class Model:
    """parts: (steps, halves) each, halves 1 or 2; one half and several steps: shared. before[e]:
    the events that stand directly in front of event e."""

    def __init__(self, parts, stages, masks, told=True):
        self.S, self.M, self.before = stages, masks, {}
        self.readers, self.tile_readers = {}, {}   # of a step's masks, of a tile
        work = []      # (first step, steps, active halves, shared)
        at = 0
        for n, halves in parts:
            shared = halves == 1 and n > 1
            work.append((at, n, halves, shared))
            at += n
        self.steps = at
        back = {}      # tile: events that give it back
        for h in (0, 1):
            self._half(h, work, back)
        self.back = back
        for v in (0, 1):
            last = []
            for J in range(at):
                use = 2 * J + v
                last = self._event(("room", use), last + self._room(use, v, told))
                last = self._event(("write", use), last)

    def _event(self, e, before):
        self.before.setdefault(e, []).extend(before)
        return [e]

    def _room(self, use, v, told):
        need, S = [], self.S
        if use >= S:
            need += self.back[use - S]
            if S % 2:      # the other loader found room for at least use + 1 - S tiles
                need += self._found(1 - v, use + 1 - S)
        if told and S % 2 == 0 and v == 0 and use >= 2 * self.M:
            need += self._found(1, use + 2 + S - 2 * self.M)
        return need

    @staticmethod
    def _found(v, tiles):      # `found` of loader v is at least this behind the room for ...
        u = tiles - 1
        if u % 2 != v:
            u += 1
        return [("room", u)] if u >= 0 else []

    def _half(self, h, work, back):
        issue, warps = [], [[] for _ in range(4)]
        for first, n, halves, shared in work:
            if not (shared or h < halves):
                continue
            steps = list(range(first + (h if shared else 0), first + n, 2 if shared else 1))
            for i, J in enumerate(steps):
                issue = self._event(("S", J, h), issue + [("write", 2 * J)])
                self.tile_readers.setdefault(2 * J, []).append(("S", J, h))
                for w in range(4):
                    warps[w] = self._event(("full", J, h, w), warps[w] + [("S", J, h)])
                    if w == 0:
                        if i > 0:
                            back.setdefault(2 * steps[i - 1] + 1, []).append(("full", J, h, 0))
                        back.setdefault(2 * J, []).append(("full", J, h, 0))
                    warps[w] = self._event(("masks", J, h, w), warps[w])
                    self.readers.setdefault(J, []).append(("masks", J, h, w))
                issue = self._event(("PV", J, h), issue + [("write", 2 * J + 1)] +
                                    [("masks", J, h, w) for w in range(4)])
                self.tile_readers.setdefault(2 * J + 1, []).append(("PV", J, h))
            if steps:
                for w in range(4):
                    warps[w] = self._event(("end", first, h, w), warps[w] + issue)
                back.setdefault(2 * steps[-1] + 1, []).append(("end", first, h, 0))

    def behind(self, e):
        seen, todo = set(), [e]
        while todo:
            for x in self.before.get(todo.pop(), ()):
                if x not in seen:
                    seen.add(x)
                    todo.append(x)
        return seen

    def unordered(self):
        bad = []
        for J in range(self.steps):
            past = self.behind(("write", 2 * J))
            old = J - self.M
            bad += [(J, r) for r in self.readers.get(old, ()) if r not in past]
            for use in (2 * J, 2 * J + 1):
                past = self.behind(("write", use))
                bad += [(use, r) for r in self.tile_readers.get(use - self.S, ()) if r not in past]
        return bad


# (steps, halves) of the parts of a block
PARTS = [
    [(1, 2)] + [(1, 1)] * 20,                 # a tile of both halves, then many of one half
    [(1, 1)] * 12 + [(1, 2), (1, 1)] * 8, [(3, 2)] + [(1, 1)] * 9 + [(2, 1)] + [(1, 1)] * 9,
    [(30, 2)], [(30, 1)], [(5, 1), (1, 2), (4, 1), (1, 1)] * 3, [(2, 1)] * 12, [(1, 2)] * 20,
    [(9, 2), (1, 1), (1, 1), (7, 1), (1, 1)] + [(1, 1)] * 12]


@pytest.mark.parametrize("parts", PARTS, ids=str)
@pytest.mark.parametrize("head_size", [64, 128])
def test_everything_that_is_overwritten_was_read(head_size, parts):
    stages, masks = constants()
    model = Model(parts, stages[head_size], masks)
    model.behind(("write", 2 * model.steps - 2))
    assert not model.unordered()


def test_the_waits_can_end():
    # nothing waits for itself
    stages, masks = constants()
    for s in stages.values():
        for parts in PARTS:
            m, state = Model(parts, s, masks), {}
            for e in list(m.before):
                stack = [(e, iter(m.before[e]))]
                while stack:
                    x, it = stack[-1]
                    state.setdefault(x, 1)
                    for y in it:
                        if state.get(y) == 1:
                            raise AssertionError((x, y))
                        if y not in state:
                            stack.append((y, iter(m.before.get(y, ()))))
                            break
                    else:
                        state[x] = 2
                        stack.pop()


def test_an_even_ring_needs_to_be_told():
    # by the key tiles alone, the warps of the half that has nothing further to do may still read
    bad = Model(PARTS[0], 12, 8, told=False).unordered()
    assert bad and all(r[0] == "masks" and r[2] == 1 for _, r in bad)
    assert not Model(PARTS[0], 5, 8, told=False).unordered()
