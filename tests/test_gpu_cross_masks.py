"""Cross attention, many rows: tiles of both halves followed by many short tiles of one half, each
with keys of its own number, so that the key masks change from step to step."""
import numpy as np
import pytest
import torch

from .step_util import CrossCase

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,bs", [(64, 16), (64, 128), (64, 20), (128, 32)])
def test_masks_of_tiles_of_one_and_of_both_halves(d, bs):
    # 2 kv heads of one query head: tiles of 256 positions; tile i goes to block i % SMs, so the
    # blocks get tiles of both kinds one after the other
    rng = np.random.default_rng(d + bs)
    nq, nk = [], []
    for _ in range(5):
        nq += [200] * 76 + [20] * 228
        nk += [int(x) for x in rng.integers(1, 129, 304)]
    c = CrossCase(95, nq, nk, num_heads=2, kv_heads=2, head_size=d, block_size=bs)
    first, lse = c.check()
    for _ in range(10):
        out, again, status = c.gpu()
        assert status == 0 and torch.equal(out, first) and torch.equal(again, lse)
