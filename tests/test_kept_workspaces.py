"""The workspaces that the cross attention's binding keeps for a thread: as many as the last
streams that it called on, given back when it asks (no GPU; see test_stream_memory)."""
import threading

from paged_kv_cache_231_gb300 import binding as B

from .test_stream_memory import Stream, cross, fake  # noqa: F401 - a fixture


def _workspaces(fake):  # noqa: F811
    return [t for t in fake.made if t.dtype is fake.uint8]


def _call_on(fake, s):  # noqa: F811
    fake.now = s
    cross()


def test_as_many_as_the_last_streams(fake):  # noqa: F811
    streams = [Stream(10 + i) for i in range(40)]
    for s in streams:
        _call_on(fake, s)
        _call_on(fake, s)
    assert len(_workspaces(fake)) == 40                  # one a stream, kept for its next call
    kept = B._OWN.__dict__
    assert list(kept) == [(0, s.cuda_stream) for s in streams[-B._OWN_STREAMS:]]
    _call_on(fake, streams[-B._OWN_STREAMS])             # the oldest is used again
    _call_on(fake, Stream(99))                           # so the one behind it goes
    _call_on(fake, streams[-B._OWN_STREAMS])
    assert len(_workspaces(fake)) == 41
    _call_on(fake, streams[-B._OWN_STREAMS + 1])
    assert len(_workspaces(fake)) == 42


def test_every_size_is_kept(fake, monkeypatch):  # noqa: F811
    # no need, whatever its size, costs an allocation a call
    for need in (1 << 10, 60 << 20, 1 << 20, 100 << 20):
        monkeypatch.setattr(B, "_cross_workspace", lambda *a: need)
        cross()
        n = len(_workspaces(fake))
        cross()
        assert len(_workspaces(fake)) == n
    assert [t.numel() for t in _workspaces(fake)] == [1 << 10, 60 << 20, 100 << 20]


def test_release(fake):  # noqa: F811
    cross()
    assert len(B._OWN.__dict__) == 1
    B.release_workspaces()
    assert not B._OWN.__dict__
    cross()
    assert len(_workspaces(fake)) == 2


def test_release_is_the_calling_threads():
    def other():
        B._OWN.__dict__[(0, 1)] = "kept"
        done.set()
        go.wait(10)
        left.append(dict(B._OWN.__dict__))

    done, go, left = threading.Event(), threading.Event(), []
    t = threading.Thread(target=other)
    t.start()
    done.wait(10)
    B.release_workspaces()
    go.set()
    t.join()
    assert left == [{(0, 1): "kept"}]
