"""Which stream and device the Python cache calls allocate on (CPU tensors stand in for a device's; no
call gets through)."""
import contextlib
import types

import pytest
import torch

import fp4_microscaling_tensor_b200 as mx
from test_cache_python_cpu import CPU, I32, cache, calls, numbers, zeros  # noqa: F401


@pytest.mark.parametrize("stream", (1234, types.SimpleNamespace(cuda_stream=1234)))
def test_scratch_for_a_raw_stream_belongs_to_the_caches_device(monkeypatch, calls, stream):  # noqa: F811
    """A stream given as its handle is one of the cache's device, not of the current one: what the call
    allocates has to be that stream's."""
    asked = []
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda handle, device=None: asked.append((handle, device)))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    mx.cache_attention(cache(), zeros(3, 5, 8, 64), zeros(3, 4, dtype=I32), numbers(), count=numbers(),
                       lse=True, stream=stream)
    assert asked == [(1234, CPU)] * 3  # out, lse and the workspace
    mx.cache_read(cache(), zeros(3, 4, dtype=I32), numbers(), None, 5, stream=stream)
    assert asked == [(1234, CPU)] * 5
    assert calls == ["mx_cache_attention", "mx_cache_read"]
