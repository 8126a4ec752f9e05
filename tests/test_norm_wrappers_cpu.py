"""Host-only tests of what the Python wrappers of the norm, SwiGLU and
checkpoint operators do before a launch: the stream they take a handle for."""
import pytest
import torch

import fp8_mixed_precision_scale_gb300 as fp8


class PoolStream:
    """torch.cuda.ExternalStream as it behaves: a handle of 0 is none given, and
    a stream of torch's pool comes back, which does not wait for the default."""

    def __init__(self, handle):
        self.cuda_stream = handle if handle else 0x5EED


class DefaultStream:
    cuda_stream = 0


@pytest.mark.parametrize("handle", [0, 0x1230])
def test_a_handle_is_the_stream_it_names(handle, monkeypatch):
    monkeypatch.setattr(torch.cuda, "ExternalStream", PoolStream)
    monkeypatch.setattr(torch.cuda, "default_stream", DefaultStream)
    monkeypatch.setattr(torch.cuda, "stream", lambda stream: stream)
    assert fp8._on(handle).cuda_stream == handle
