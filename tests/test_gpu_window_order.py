"""Causal attention over cumulative lengths that do not ascend: rows of exactly one sound sequence get
its result, rows of none output 0 and lse -inf; rows that two claim are either's."""
import numpy as np
import pytest
import torch

from paged_kv_cache_231_gb300 import binding as B

from .cache_util import CausalCase
from .step_util import cross_bound, wide

pytestmark = pytest.mark.gpu

# in units of n rows, of 12 (and 3 rows behind them); a sequence's table is filled for 3 units, so no
# sound one holds more: what lies behind is NaN
ORDERS = {"falls and rises": (0, 1, 2, 1, 4), "begins late": (1, 2, 0, 1, 3),
          "empty in front": (5, 5, 6, 2, 4), "past the end": (0, 1, 20, 3, 4),
          "below zero": (-1, 1, 2, 2, 2), "all fall": (4, 3, 2, 1, 0),
          "gap in the middle": (9, 10, 0, 1, 3), "two overlap": (0, 1, 4, 2, 5),
          "one holds another's": (6, 0, 1, 0, 3)}


def check(c, cu, prefix=False, **kw):
    c.cu = np.array(cu, np.int32)
    T = c.q.shape[0]
    claims = np.zeros(T, int)
    for lo, hi in zip(cu, cu[1:]):
        if 0 <= lo <= hi <= T:
            claims[lo:hi] += 1
    out, lse, status = c.gpu(prefix=prefix, **kw)
    ref, rlse, size, reach, want = c.oracle()
    assert status == want
    got, lse = wide(out).reshape(ref.shape), wide(lse)
    none, one = claims == 0, claims == 1
    assert not got[none].any() and np.isneginf(lse[none]).all()
    assert not np.isnan(got).any() and not np.isnan(lse).any()
    values = float(c.v[~torch.isnan(c.v)].abs().double().mean())
    n = max(len(j) for j in c.seen) + 1
    # as CausalCase.check
    tol, tol_lse = cross_bound(c.t, ref, rlse, size * (1 + 2.0 ** -10 * prefix), reach, n, values)
    tol = tol + 2.0 ** -19 * size * prefix
    assert (np.abs(got - ref) <= tol)[one].all()
    assert (np.abs(lse[one] - rlse[one]) <= tol_lse[one] + 2.0 ** -20 * prefix).all()


@pytest.mark.parametrize("order", list(ORDERS))
@pytest.mark.parametrize("n", [1, 2, 7, 70, 300])
@pytest.mark.parametrize("window,sinks", [(0, 0), (25, 3)])
def test_window(order, n, window, sinks):
    c = CausalCase(1, [3 * n] * 4, [120, 95, 100, 130], window=window, sinks=sinks, pad=3)
    check(c, [n * x for x in ORDERS[order]])


@pytest.mark.parametrize("sharing", [0, 1])
@pytest.mark.parametrize("order", list(ORDERS))
@pytest.mark.parametrize("n", [1, 7, 70])
def test_behind_a_prefix(order, n, sharing):
    c = CausalCase(2, [3 * n] * 4, [120, 95, 100, 130], groups=[(2, 80), (2, 96)], pad=3)
    B.pkv_testing_prefix_sharing(sharing)
    try:
        check(c, [n * x for x in ORDERS[order]], prefix=True)
    finally:
        B.pkv_testing_prefix_sharing()
