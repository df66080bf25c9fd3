"""Which stream the memory that the attention, block-sparse and combine calls make comes from (no
GPU; see test_stream_memory)."""
import types

import pytest
import torch

from paged_kv_cache_231_gb300 import binding as B

from .test_stream_memory import Stream, Tensor, fake  # noqa: F401 - a fixture

i32, f16, f32 = torch.int32, torch.float16, torch.float32


@pytest.fixture
def lib(fake, monkeypatch):  # noqa: F811
    def entry(name):
        def call(*a):
            fake.calls.append((name, a))
            return 0
        return call

    names = ("pkv_paged_attention", "pkv_sparse_attention_partials", "pkv_combine_partials")
    monkeypatch.setattr(B, "load_library",
                        lambda: types.SimpleNamespace(**{n: entry(n) for n in names}))
    monkeypatch.setattr(B, "_check_paged_tensors", lambda *a: None)
    for n in names[:2]:
        monkeypatch.setattr(B, n + "_workspace_size", lambda a: 1 << 20)
    return fake


def attention(**kw):
    pool, rows = Tensor((4, 8, 2, 64), f16), Tensor((3, 128), f16)
    return [B.pkv_paged_attention(Tensor((3, 256), f16), rows, rows, pool, pool,
                                  Tensor((3,), i32), Tensor((2,), i32), Tensor((2, 4), i32),
                                  num_heads=4, kv_num_heads=2, **kw)]


def partials(**kw):
    pages = Tensor((6, 2, 8, 64), f32)
    return B.pkv_sparse_attention_partials(Tensor((3, 4, 64), f32), pages, pages,
                                           Tensor((5, 4), i32), Tensor((2, 3), i32), qhead=4,
                                           block_size=8, page_size=8, pages_per_block=1,
                                           softmax_scale=0.1, **kw)


def combine(**kw):
    return B.pkv_combine_partials(Tensor((8, 64), f32), Tensor((8,), f32), Tensor((8,), f32),
                                  num_segments=2, lanes=2, uniform_count=2, **kw)[:1]


CALLS = pytest.mark.parametrize("call", [attention, partials, combine])


@CALLS
@pytest.mark.parametrize("capturing", [False, True])
def test_another_stream(lib, call, capturing):
    side = Stream(7, capturing)
    returned = call(stream=side)
    assert lib.made and all(t.made_on is side and t.capturing == capturing for t in lib.made)
    for t in lib.made:
        assert t.recorded == ([lib.main] if any(t is r for r in returned) else [])
    assert lib.calls[0][1][-1] == 7 and lib.now is lib.main


@CALLS
def test_the_current_stream(lib, call):
    call()
    assert lib.made and all(t.made_on is lib.main and not t.recorded for t in lib.made)
    assert lib.calls[0][1][-1] == 1
