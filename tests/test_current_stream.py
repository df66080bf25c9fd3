"""The step operators' calls go to the current stream also where torch has no short way to its
handle (no GPU; see test_stream_memory)."""
import types

import pytest

from .test_stream_memory import CALLS, Stream, append, cross, fake, schedule  # noqa: F401


@CALLS
@pytest.mark.parametrize("short_way", [True, False])
def test_handle_of_the_current_stream(fake, call, short_way):  # noqa: F811
    if not short_way:
        fake._C = types.SimpleNamespace()
    fake.now = Stream(31)
    call()
    call(stream=Stream(32))
    assert [a[-1] for _, a in fake.calls] == [31, 32]
