"""The list of caches of pkv_paged_fork (no GPU)."""
import pytest
import torch

from paged_kv_cache_231_gb300 import binding as B


def test_one_tensor_is_no_list_of_caches():
    # it has a length and items too: each of its blocks would pass for a cache of its own
    z = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(TypeError, match="caches: a list of tensors"):
        B.pkv_paged_fork(z(2), z(2), z(2, 4), torch.zeros(8, 16, 2, 64))
