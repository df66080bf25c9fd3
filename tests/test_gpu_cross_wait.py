"""The give-up path of the cross attention's bounded waits (the kernel for many rows): with
the first key tile withheld the call returns with PKV_DEV_TIMEOUT set, and the next call is
right again."""
import pytest

from paged_kv_cache_231_gb300 import binding as B

from .step_util import CrossCase

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("head_size,block_size", [(128, 16), (64, 32)])
def test_wait_gives_up_then_recovers(head_size, block_size):
    c = CrossCase(31, [200, 1, 90], [300, 70, 1000], num_heads=4, kv_heads=2,
                  head_size=head_size, block_size=block_size)
    B.pkv_testing_wait_limit(4096, True)
    try:
        status = c.gpu()[2]
    finally:
        B.pkv_testing_wait_limit()
    assert status == B.DEV_TIMEOUT
    c.check()
