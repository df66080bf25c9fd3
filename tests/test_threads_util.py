"""The helper for calls of several threads (no GPU)."""
import threading

import pytest

from .threads_util import at_once


def test_results_in_order_and_side_by_side():
    here = threading.Barrier(3, timeout=20)     # nobody goes on before all three run
    assert at_once([lambda i=i: (here.wait() >= 0, i)[1] for i in range(3)]) == [0, 1, 2]


def test_what_a_thread_raises_is_raised():
    def refuse():
        raise RuntimeError("refused")
    with pytest.raises(RuntimeError, match="refused"):
        at_once([lambda: 1, refuse])
