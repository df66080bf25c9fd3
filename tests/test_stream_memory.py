"""Which stream the memory that the binding makes for a call comes from. No GPU: the binding runs
over a stand-in for torch that notes the stream every tensor is asked for on."""
import contextlib
import types

import pytest
import torch

from paged_kv_cache_231_gb300 import binding as B

i32, f16 = torch.int32, torch.float16


class Tensor:
    def __init__(self, shape, dtype, made_on=None, capturing=False):
        self.shape = tuple(shape) if isinstance(shape, (tuple, list)) else (shape,)
        self.dtype, self.made_on, self.capturing = dtype, made_on, capturing
        self.recorded, self.device, self.is_cuda = [], "cuda:0", True

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 4096

    def record_stream(self, stream):
        self.recorded.append(stream)


class Stream:
    device_index = 0

    def __init__(self, handle, capturing=False):
        self.cuda_stream, self.capturing = handle, capturing


class FakeTorch:
    def __init__(self):
        self.main = self.now = Stream(1)
        self.made = []
        for name in ("float16", "bfloat16", "float32", "int32", "uint8"):
            setattr(self, name, getattr(torch, name))
        self.cuda = types.SimpleNamespace(
            current_device=lambda: 0, current_stream=lambda device=None: self.now,
            is_current_stream_capturing=lambda: self.now.capturing, stream=self.stream)
        self._C = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda d: self.now.cuda_stream)

    @contextlib.contextmanager
    def stream(self, s):
        before, self.now = self.now, s
        try:
            yield
        finally:
            self.now = before

    def empty(self, shape, dtype=None, device=None):
        t = Tensor(shape, dtype, self.now, self.now.capturing)
        self.made.append(t)
        return t


@pytest.fixture
def fake(monkeypatch):
    f = FakeTorch()
    f.calls = []
    monkeypatch.setattr(B, "_torch", lambda: f)
    monkeypatch.setattr(B, "_step_call", lambda name, *a: f.calls.append((name, a)))
    monkeypatch.setattr(B, "_cross_workspace", lambda *a: 1 << 20)
    monkeypatch.setattr(B, "_OWN", types.SimpleNamespace())
    return f


def schedule(**kw):
    return B.pkv_paged_schedule(Tensor((2,), i32), Tensor((2,), i32), Tensor((2, 4), i32),
                                num_blocks=8, block_size=4, num_tokens=5, **kw)


def append(**kw):
    rows = Tensor((3, 256), f16)
    return [B.pkv_paged_append_rotary_axes(rows, Tensor((3, 128), f16), Tensor((3, 128), f16),
                                           Tensor((4, 8, 2, 64), f16), Tensor((4, 8, 2, 64), f16),
                                           Tensor((3,), i32), None, num_heads=4, kv_num_heads=2,
                                           **kw)]


def cross(**kw):
    pool = Tensor((4, 8, 2, 64), f16)
    return [B.pkv_cross_attention(Tensor((3, 256), f16), pool, pool, Tensor((3,), i32),
                                  Tensor((2,), i32), Tensor((2, 4), i32), num_heads=4,
                                  kv_num_heads=2, **kw)]


CALLS = pytest.mark.parametrize("call", [schedule, append, cross])


@CALLS
@pytest.mark.parametrize("capturing", [False, True])
def test_another_stream(fake, call, capturing):
    side = Stream(7, capturing)
    returned = call(stream=side)
    assert fake.made and all(t.made_on is side for t in fake.made)
    assert all(t.capturing == capturing for t in fake.made)   # a captured call's: the graph's
    for t in fake.made:   # what the caller gets is used on the current stream too
        assert t.recorded == ([fake.main] if any(t is r for r in returned) else [])
    assert fake.calls[0][1][-1] == 7 and fake.now is fake.main


@CALLS
@pytest.mark.parametrize("named", [False, True])
def test_the_current_stream(fake, call, named):
    call(**(dict(stream=fake.main) if named else {}))
    assert fake.made and all(t.made_on is fake.main and not t.recorded for t in fake.made)
    assert fake.calls[0][1][-1] == 1
