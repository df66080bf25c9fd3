"""The operators around the paged cache called by threads that share a stream, and by threads on
streams of their own: every call gives its result, bit for bit, and none is refused."""
import pytest
import torch

from paged_kv_cache_231_gb300 import binding as B

from .test_gpu_cache_edges import Calls
from .threads_util import at_once

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[0, 1], autouse=True)
def sharing(request):
    B.pkv_testing_prefix_sharing(request.param)
    yield
    B.pkv_testing_prefix_sharing()


def bits(x):
    return x.view(torch.int16)


@pytest.mark.parametrize("streams", [1, 2, 4])
def test_threads(streams):
    calls = [Calls(20 + i) for i in range(4)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    made = [torch.cuda.Stream() for _ in range(streams)]

    def work(i):
        with torch.cuda.stream(made[i % streams]):
            got = [calls[i]() for _ in range(25)]
        torch.cuda.synchronize()
        return got

    results = at_once([lambda i=i: work(i) for i in range(4)])
    for got, expected in zip(results, want):
        assert len(got) == 25
        for g in got:
            assert len(g) == len(expected) == 5
            assert all(torch.equal(bits(x), bits(y)) for x, y in zip(g, expected))
