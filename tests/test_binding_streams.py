"""The stream handle that the binding passes to the library, without a GPU."""
import types

import pytest

import context_attention_metadata_gb300 as M


@pytest.mark.parametrize("index", [None, 3])
def test_current_stream_with_and_without_the_direct_call(monkeypatch, index):
    """Where this torch has no direct call for the current stream's handle, the public one is
    taken; a stream that is given is used as it is."""
    stream = types.SimpleNamespace(cuda_stream=77)
    asked = []
    cuda = types.SimpleNamespace(current_device=lambda: 1,
                                 current_stream=lambda i: asked.append(i) or stream)
    fake = types.SimpleNamespace(_C=types.SimpleNamespace(), cuda=cuda)
    assert M._raw_stream(fake, None, index) == 77 and asked == [index]
    fake._C._cuda_getCurrentRawStream = lambda i: 100 + i
    assert M._raw_stream(fake, None, index) == 100 + (1 if index is None else index)
    assert M._raw_stream(fake, stream, index) == 77 and asked == [index]
